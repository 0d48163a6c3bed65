"""How the decode-step operators are called from Python: empty calls, shapes that are
refused, the status-returning forms, several streams and several host threads."""
import threading

import pytest
import torch

import deterministic_fixed_order_gb300 as df
from test_gpu_attn import BF16, F16, F32, Append, Decode, gen, join_inputs, randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

A = df.attention
S = df.STATUS


def empty(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda")


# ------------------------------------------------------------------ nothing to do

@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_calls_without_rows_do_nothing(dtype):
    cache = df.PagedCache(empty(4, 16, 2, 64, dtype=dtype), empty(4, 16, 2, 64, dtype=dtype))
    k0 = cache.k.fill_(3).clone()
    cache.v.fill_(4)
    rope = df.Rope(torch.ones((10, 64), device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    long = empty(0, dtype=torch.int64)
    df.detfold_kv_append(cache, empty(0, 2, 64, dtype=dtype), empty(0, 2, 64, dtype=dtype), long)
    df.detfold_kv_append(cache, empty(0, 2, 64, dtype=dtype), empty(0, 2, 64, dtype=dtype), long, rope=rope,
                         positions=long, q=empty(0, 8, 64, dtype=dtype), q_out=empty(0, 8, 64, dtype=dtype),
                         status=status)
    for cols in (0, 4):
        df.detfold_attn_decode(empty(0, 8, 64, dtype=dtype), empty(0, 8, 64, dtype=dtype), cache,
                               empty(0, cols, dtype=torch.int32), empty(0, dtype=torch.int32), 0, 0.125, status=status)
    df.detfold_attn_decode(empty(0, 8, 64, dtype=dtype), empty(0, 8, 64, dtype=dtype), cache,
                           empty(0, 4, dtype=torch.int32), empty(0, dtype=torch.int32), 64, 0.125, window=7,
                           lse=empty(0, 8, dtype=F32), status=status)
    for shape in ((0,), (0, 5), (5, 0)):
        df.detfold_attn_join(empty(*shape, 64, dtype=dtype), [empty(*shape, 64, dtype=dtype) for _ in range(3)],
                             [empty(*shape, dtype=F32) for _ in range(3)], lse=empty(*shape, dtype=F32))
    torch.cuda.synchronize()
    assert int(status) == 0 and torch.equal(cache.k, k0) and bool((cache.v == 4).all())


def test_sequences_without_a_table():
    # max_len 0: no page is looked up, so the table may have no columns
    cache = df.PagedCache(empty(4, 16, 2, 64), empty(4, 16, 2, 64))
    q, out, lse = randn(gen(1), (3, 8, 64), BF16), empty(3, 8, 64), empty(3, 8, dtype=F32)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    df.detfold_attn_decode(out, q, cache, empty(3, 0, dtype=torch.int32), lens, 0, 0.125, lse=lse)
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())


def test_what_is_wrong_without_rows_is_refused_all_the_same():
    cache = df.PagedCache(empty(4, 16, 2, 64), empty(4, 16, 2, 64))
    none = empty(0, dtype=torch.int32)
    for kw, code in ((dict(heads=7), "DETFOLD_ERR_ARG"), (dict(window=-1), "DETFOLD_ERR_ARG"),
                     (dict(max_len=65), "DETFOLD_ERR_LEN"), (dict(max_len=-1), "DETFOLD_ERR_LEN")):
        a = {**dict(heads=8, window=0, max_len=64), **kw}
        with pytest.raises(df.DetfoldError) as e:
            df.detfold_attn_decode(empty(0, a["heads"], 64), empty(0, a["heads"], 64), cache,
                                   empty(0, 4, dtype=torch.int32), none, a["max_len"], 0.125, window=a["window"])
        assert e.value.status == S[code], kw
    with pytest.raises(ValueError):
        df.detfold_kv_append(cache, empty(0, 2, 64), empty(0, 3, 64), empty(0, dtype=torch.int64))
    with pytest.raises(df.DetfoldError) as e:
        df.detfold_attn_join(empty(0, 64), [], [])
    assert e.value.status == S["DETFOLD_ERR_WORLD"]


# ------------------------------------------------------------------ shapes

def test_join_takes_parts_of_its_output_s_shape_only():
    parts, lses = join_inputs(BF16, 3, (6, 4), 8)
    out, lse = torch.empty_like(parts[0]), torch.empty_like(lses[0])
    df.detfold_attn_join(out, parts, lses, lse=lse)
    for name, bad in (("parts", dict(parts=[parts[0], parts[1].view(4, 6, 8), parts[2]])),
                      ("parts", dict(parts=[parts[0], parts[1], parts[2].view(6, 8, 4)])),
                      ("parts", dict(parts=[parts[0].view(24, 8)] + parts[1:])),
                      ("lses", dict(lses=[lses[0].view(4, 6)] + lses[1:])),
                      ("lses", dict(lses=lses[:2] + [lses[2].view(24)])),
                      ("lse", dict(lse=torch.empty((4, 6), device="cuda")))):
        with pytest.raises(ValueError, match="^" + name + ":"):
            df.detfold_attn_join(**{**dict(out=out, parts=parts, lses=lses, lse=lse), **bad})


def test_decode_takes_an_lse_of_a_value_a_query_head_only():
    d = Decode(BF16, [40, 3], 8, 2, 64, 16)
    out = torch.empty_like(d.q)
    df.detfold_attn_decode(out, d.q, d.cache, d.table, d.lens, d.max_len, 1.0, lse=torch.empty((2, 8), device="cuda"))
    for shape in ((8, 2), (16,), (2, 8, 1)):
        with pytest.raises(ValueError, match="^lse:"):
            df.detfold_attn_decode(out, d.q, d.cache, d.table, d.lens, d.max_len, 1.0,
                                   lse=torch.empty(shape, device="cuda"))


# ------------------------------------------------------------------ the status-returning forms

def test_status_forms_return_what_the_others_raise():
    d = Decode(BF16, [40, 3], 8, 2, 64, 16)
    want, wlse = d.run()
    out, lse = torch.empty_like(d.q), torch.empty((2, 8), device="cuda")
    args = (d.q, d.cache, d.table, d.lens)
    assert A.status_attn_decode(out, *args, d.max_len, d.scale, lse=lse) == S["DETFOLD_OK"]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert A.status_attn_decode(out, *args, 1000, d.scale) == S["DETFOLD_ERR_LEN"]
    assert A.status_attn_decode(d.q, *args, d.max_len, d.scale) == S["DETFOLD_ERR_OVERLAP"]
    with pytest.raises(TypeError):
        A.status_attn_decode(out.half(), *args, d.max_len, d.scale)

    a, b = Append(BF16, 20, 4, 2, 64, 64, False), Append(BF16, 20, 4, 2, 64, 64, False)
    qa, qb = torch.empty((20, 4, 64), dtype=BF16, device="cuda"), torch.empty((20, 4, 64), dtype=BF16, device="cuda")
    df.detfold_kv_append(a.cache, a.nk, a.nv, a.slots, rope=a.rope, positions=a.positions, q=a.q, q_out=qa)
    assert A.status_kv_append(b.cache, b.nk, b.nv, b.slots, rope=b.rope, positions=b.positions, q=b.q, q_out=qb) == 0
    torch.cuda.synchronize()
    assert torch.equal(qa, qb) and torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert A.status_kv_append(a.cache, a.k[0, :6], a.nv[:6], a.slots[:6]) == S["DETFOLD_ERR_OVERLAP"]

    parts, lses = join_inputs(BF16, 3, (5,), 64)
    one, two = torch.empty_like(parts[0]), torch.empty_like(parts[0])
    df.detfold_attn_join(one, parts, lses)
    assert A.status_attn_join(two, parts, lses) == S["DETFOLD_OK"]
    torch.cuda.synchronize()
    assert torch.equal(one, two)
    assert A.status_attn_join(two, [], []) == S["DETFOLD_ERR_WORLD"]


# ------------------------------------------------------------------ at the same time

def test_calls_at_the_same_time_on_two_streams():
    # a workspace and outputs each; every call's bits are those of the call alone
    jobs = [Decode(BF16, [9000, 40, 1200], 32, 8, 128, 16, seed=1), Decode(F32, [2500, 0, 700, 90], 8, 8, 64, 16, seed=2)]
    want = [d.run() for d in jobs]
    spaces = [torch.empty(df.detfold_attn_decode_workspace_bytes(d.cache, d.q.shape[0], d.q.shape[1], d.max_len) + 16,
                          dtype=torch.uint8, device="cuda") for d in jobs]
    outs = [[(torch.empty_like(d.q), torch.empty(d.q.shape[:2], device="cuda")) for _ in range(25)] for d in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()  # what the streams use is there
    for i in range(25):
        for d, ws, out, stream in zip(jobs, spaces, outs, streams):
            df.detfold_attn_decode(out[i][0], d.q, d.cache, d.table, d.lens, d.max_len, d.scale, lse=out[i][1],
                                   workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for got, (o, s) in zip(outs, want):
        assert all(torch.equal(a, o) and torch.equal(b, s) for a, b in got)


def test_calls_from_several_host_threads():
    # a step of each thread's own: append, attention and join, on a stream of its own
    def job(seed):
        d = Decode(BF16, [1500, 40 + seed], 8, 2, 64, 16, seed=seed)
        a = Append(BF16, 33, 8, 2, 64, 64, False, seed=seed)
        parts, lses = join_inputs(BF16, 3, (50,), 64, seed=seed)
        ws = torch.empty(df.detfold_attn_decode_workspace_bytes(d.cache, 2, 8, d.max_len) + 16, dtype=torch.uint8,
                         device="cuda")
        return d, a, parts, lses, ws

    def step(j, stream):
        d, a, parts, lses, ws = j
        with torch.cuda.stream(stream):
            out, q_out, joined = torch.empty_like(d.q), torch.empty(a.q.shape, dtype=BF16, device="cuda"), torch.empty_like(parts[0])
            df.detfold_kv_append(a.cache, a.nk, a.nv, a.slots, rope=a.rope, positions=a.positions, q=a.q, q_out=q_out)
            df.detfold_attn_decode(out, d.q, d.cache, d.table, d.lens, d.max_len, d.scale, workspace=ws)
            df.detfold_attn_join(joined, parts, lses)
        return out, q_out, joined

    jobs = [job(1 + t) for t in range(4)]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    want = [step(j, s) for j, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(t):
        try:
            got[t] = [step(jobs[t], streams[t]) for _ in range(20)]
            streams[t].synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for t in range(4):
        for one in got[t]:
            assert all(torch.equal(x, y) for x, y in zip(one, want[t])), t

"""kvq_chunk_attention against the formula in 64 bits over the values the pool
holds: ragged chunks, single tokens, caps, distance biases, windows, prefixes,
empty rows, unwritten slots, missing pages, bad ranges, strides and streams."""
import ctypes

import numpy as np
import pytest
import torch

from _helpers import MODE_NAMES, TENSOR_SCALED, guarded, kvq
from test_norm_rope_read import pool_values

ROWS = [m for m in MODE_NAMES if not m.startswith("kvarn")]


def build(mode, io, H, D, lens, seed=1, gain=1.0, v_gain=None):
    """A cache holding sequences of these lengths on scattered pages; slots past a sequence's end stay 0xFF (NaN
    patterns).  Returns (cache, block_table numpy, values [2][pages][16][H][D])."""
    K = kvq()
    rng = np.random.default_rng(seed)
    dt = torch.float16 if io == "f16" else torch.float32
    per = [(n + 15) // 16 for n in lens]
    pages = sum(per) + 2
    cfg = K.make_config(pages, 16, H, D, mode, dt)
    pool = guarded(K.kvq_cache_bytes(cfg), torch.uint8, fill=0xFF, name="pool")
    cache = K.kvq_cache_alloc(cfg, pool)
    ks = vs = 1.0
    vg = gain if v_gain is None else v_gain
    if mode in TENSOR_SCALED:
        div = 448.0 if mode == "fp8_per_tensor" else 2688.0
        ks, vs = (float(np.float32(5.0 * g / div)) for g in (gain, vg))
        K.kvq_cache_set_tensor_scales(cache, ks, vs)
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(per + [1]) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        table[b, :per[b]] = perm[at:at + per[b]]
        at += per[b]
        if not n:
            continue
        k, v = (torch.from_numpy(rng.standard_normal((n, H, D)) * g).to(dt).cuda() for g in (gain, vg))
        t = np.arange(n)
        slots = torch.from_numpy((table[b, t // 16] * 16 + t % 16).astype(np.int32)).cuda()
        K.kvq_quantize_write(cache, k, v, slots)
    torch.cuda.synchronize()
    vals = pool_values(mode, pool.cpu().numpy(), pages, H, D, ks, vs)
    return cache, table, vals


def formula(vals, table, q, cu, lens, scale, cap=0.0, slopes=None, window=0, prefix=None, missing=()):
    """[total_q][Hq][D] in 64 bits; NaN rows where no sequence has the row."""
    H = vals.shape[3]
    Hq, D = q.shape[1:]
    out = np.full(q.shape, np.nan)
    for b, n in enumerate(lens):
        t = np.arange(n)
        k, v = vals[:, table[b, t // 16], t % 16] if n else np.zeros((2, 0, H, D))
        here = np.array([(table[b, x // 16] not in missing) for x in t], bool)
        m = cu[b + 1] - cu[b]
        for i in range(m):
            p = n - m + i
            see = t <= p
            if window:
                see &= t > p - window
            if prefix is not None:
                see |= t < prefix[b]
            see &= here & (p >= 0)
            for h in range(Hq):
                if not see.any():
                    out[cu[b] + i, h] = 0.0
                    continue
                s = scale * (k[see, h // (Hq // H)] @ q[cu[b] + i, h].astype(np.float64))
                if cap:
                    s = cap * np.tanh(s / cap)
                if slopes is not None:
                    s = s - float(slopes[h]) * np.abs(p - t[see])
                w = np.exp(s - s.max())
                out[cu[b] + i, h] = w @ v[see, h // (Hq // H)] / w.sum()
    return out


def tolerance(want, vmax, smax, n, dt, f32):
    """Of an output: its own rounding (eps / 2 of it), and the weights' error times the largest value that can enter.
    A weight errs by its exponent's (scores of magnitude smax log2 units held in fp32: 4 roundings of the score and
    its fp32 sum over 128 channels) and by its own rounding: fp16 weights 2^-11 (a half-ulp each, fp16 outputs only),
    else 2^-21 of the hi + lo pair; the sums over n tokens err by 2^-23 a term at most in relation to their size."""
    eps = torch.finfo(dt).eps / 2
    weight = (2.0 ** -21 if f32 else 2.0 ** -11) + 12 * 2.0 ** -23 * max(smax, 1.0) + min(n, 64) * 2.0 ** -23
    return eps * np.abs(want) + 2 * weight * vmax + 2.0 ** -24


def run(cache, table, q, cu, lens, out_dtype, max_q=None, max_n=None, fill=7.0, **kw):
    K = kvq()
    out = guarded(q.shape, out_dtype, fill=fill, name="out")
    max_q = int(np.diff(cu).max()) if max_q is None else max_q
    max_n = max(lens) if max_n is None else max_n
    _, _, wsb = K.kvq_chunk_plan(cache, q.shape[0], len(lens), q.shape[1], max_q_len=max_q, max_seq_len=max_n,
                                 window=kw.get("window", 0), has_prefix=kw.get("prefix_lens") is not None)
    ws = guarded(max(wsb // 4, 1), torch.float32, fill=float("nan"), name="workspace")
    ints = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    K.kvq_chunk_attention(cache, q, ints(cu), ints(table), ints(lens), out, max_q_len=max_q, max_seq_len=max_n,
                          workspace=ws, **kw)
    torch.cuda.synchronize()
    return out


def check(mode, io, out, H, G, D, qlens, lens, cap=0.0, alibi=False, window=0, prefix=False, seed=1, gain=1.0,
          v_gain=None, scale=None, tail_rows=2, max_n=None):
    cache, table, vals = build(mode, io, H, D, lens, seed, gain, v_gain)
    rng = np.random.default_rng(seed + 100)
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    dt = torch.float16 if io == "f16" else torch.float32
    odt = torch.float16 if out == "f16" else torch.float32
    q = torch.from_numpy(rng.standard_normal((cu[-1] + tail_rows, H * G, D))).to(dt).cuda()
    scale = D ** -0.5 if scale is None else scale
    slopes = (2.0 ** (-8.0 * np.arange(1, H * G + 1) / (H * G))).astype(np.float32) if alibi else None
    pre = np.array([rng.integers(0, n + 5) for n in lens], np.int32) if prefix else None
    got = run(cache, table, q, cu, lens, odt, softmax_scale=scale, logit_cap=cap, window=window, max_n=max_n,
              alibi_slopes=None if slopes is None else torch.from_numpy(slopes).cuda(),
              prefix_lens=None if pre is None else torch.from_numpy(pre).cuda())
    assert kvq().kvq_cache_read_errors(cache) == 0
    want = formula(vals, table, q.cpu().numpy(), cu, lens, scale, cap, slopes, window,
                   None if pre is None else np.minimum(pre, lens))
    g = got.double().cpu().numpy()
    rows = ~np.isnan(want[:, 0, 0])
    assert (g[~rows] == 7.0).all(), "rows of no sequence were written"
    fin = vals[1][np.isfinite(vals[1])]
    smax = 1.4427 * (cap if cap else scale * np.sqrt(D) * np.abs(vals[0][np.isfinite(vals[0])]).max() * 4)
    tol = tolerance(want[rows], np.abs(fin).max(), smax, max(lens), odt, odt == torch.float32)
    err = np.abs(g[rows] - want[rows])
    assert np.isfinite(g[rows]).all() and (err <= tol).all(), f"worst {np.max(err / tol):.2f} of the tolerance"
    return cache


# ---------------------------------------------------------------- refusals (CPU)
def test_refusals_before_device_work():
    K = kvq()
    lib = K.lib()
    assert lib.kvq_chunk_plan(None, 1, 1, 8, 1, 16, None, None, None) == 1
    assert lib.kvq_chunk_attention(None, None, 1, None, None, 1, None, 1, 8, 1, 16, 4, 0.1, None, None, 0, None, 0,
                                   None) == 1


# ---------------------------------------------------------------- values
@pytest.mark.gpu
@pytest.mark.parametrize("io,out", [("f16", "f16"), ("f16", "f32"), ("f32", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("mode", ROWS)
@pytest.mark.parametrize("D", [32, 128])
def test_ragged_batch(mode, io, out, D):
    # a prompt, a chunk behind a context, a single token, an empty chunk, more queries than tokens, an empty sequence
    check(mode, io, out, 2, 3, D, [40, 33, 1, 0, 9, 2], [40, 150, 77, 30, 5, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("io,out", [("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("mode", ["int8_per_token_head", "nvfp4"])
@pytest.mark.parametrize("opts", [dict(cap=5.0), dict(alibi=True), dict(window=1), dict(window=37), dict(prefix=True),
                                  dict(prefix=True, window=20), dict(cap=2.0, window=64, alibi=True, prefix=True)],
                         ids=str)
def test_options(mode, io, out, opts):
    check(mode, io, out, 1, 8, 128, [70, 1, 20], [70, 260, 301], **opts)
    check(mode, io, out, 2, 1, 32, [70, 1, 20], [70, 260, 301], **opts)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ROWS)
@pytest.mark.parametrize("opts", [dict(), dict(cap=5.0, alibi=True), dict(window=33), dict(prefix=True, window=16)], ids=str)
def test_single_tokens(mode, opts):
    check(mode, "f16", "f16", 2, 4, 128, [1, 1, 0, 1, 1, 1], [1, 16, 40, 0, 300, 2000], **opts)
    check(mode, "f32", "f32", 1, 2, 32, [1, 1, 0, 1], [1, 17, 40, 333], **opts)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int8_per_token_head", "fp8_per_token_head", "int4_per_token_head", "fp8_per_tensor"])
@pytest.mark.parametrize("qlens,lens", [([300, 5], [300, 400]), ([1, 1], [700, 20])])
def test_magnitudes(mode, qlens, lens):
    """Small and large keys and values: the weights keep their bits whatever the scales beside them."""
    check(mode, "f16", "f16", 1, 4, 128, qlens, lens, gain=0.02, v_gain=2e-3, scale=50.0)
    check(mode, "f16", "f32", 1, 4, 128, qlens, lens, gain=30.0, v_gain=3e3, scale=2e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int8_per_token_head", "nvfp4"])
def test_values_that_grow_and_vanish(mode):
    """A sequence whose first tokens hold zero values and whose later ones grow by orders of magnitude."""
    K = kvq()
    n, H, D = 900, 1, 128
    cache, table, _ = build(mode, "f16", H, D, [n])
    rng = np.random.default_rng(9)
    grow = np.concatenate([np.zeros(200), 10.0 ** np.linspace(-3, 3, n - 200)])
    k = torch.from_numpy(rng.standard_normal((n, H, D))).half().cuda()
    v = torch.from_numpy(rng.standard_normal((n, H, D)) * grow[:, None, None]).half().cuda()
    t = np.arange(n)
    K.kvq_cache_set_tensor_scales(cache, 5.0 / 2688.0, 5e3 / 2688.0)
    K.kvq_quantize_write(cache, k, v, torch.from_numpy((table[0, t // 16] * 16 + t % 16).astype(np.int32)).cuda())
    vals = pool_values(mode, cache.pool.cpu().numpy(), cache.cfg.num_pages, H, D, 5.0 / 2688.0, 5e3 / 2688.0)
    cu = np.array([0, n], np.int32)
    q = torch.from_numpy(rng.standard_normal((n, 2, D))).half().cuda()
    got = run(cache, table, q, cu, [n], torch.float16).double().cpu().numpy()
    want = formula(vals, table, q.cpu().numpy(), cu, [n], D ** -0.5)
    for i in range(n):  # a row's tolerance goes by the values it sees
        vmax = np.abs(vals[1][table[0, t[:i + 1] // 16], t[:i + 1] % 16]).max()
        tol = tolerance(want[i], vmax, 10.0, n, torch.float16, False)
        assert (np.abs(got[i] - want[i]) <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("qlens,lens,heads", [([1], [1], (1, 1)), ([2], [2], (1, 8)), ([129], [129], (1, 1)),
                                              ([257, 31], [1111, 31], (2, 7)), ([64, 1, 1, 1], [5000, 4000, 3, 17], (1, 8)),
                                              ([3] * 40, list(range(3, 123, 3)), (3, 5))])
def test_sizes(qlens, lens, heads):
    check("fp8_per_token_head", "f16", "f16", heads[0], heads[1], 128, qlens, lens)
    check("nvfp4", "f16", "f16", heads[0], heads[1], 128, qlens, lens, window=100)


@pytest.mark.gpu
@pytest.mark.parametrize("qlens", [[20, 30], [1, 1]])
def test_missing_pages_and_bad_ranges(qlens):
    K = kvq()
    lens = [100, 90]
    cache, table, vals = build("int8_per_token_head", "f16", 1, 128, lens)
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    q = torch.randn(cu[-1], 4, 128, device="cuda").half()
    bad = table.copy()
    bad[0, 2] = -1
    bad[1, 1] = cache.cfg.num_pages
    got = run(cache, bad, q, cu, lens, torch.float32)
    assert K.kvq_cache_read_errors(cache) == 0x2
    hole = table.copy()
    want = formula(vals, hole, q.cpu().numpy(), cu, lens, 128 ** -0.5, missing=(table[0, 2], table[1, 1]))
    assert np.abs(got.double().cpu().numpy() - want).max() < 1e-4
    # sequence 1's range runs past the batch: it is skipped, its rows stay
    wrong = cu.copy()
    wrong[2] += 1
    got = run(cache, table, q, wrong, lens, torch.float32, max_q=max(qlens) + 1)
    assert K.kvq_cache_read_errors(cache) == 0x100
    assert (got[cu[1]:] == 7.0).all()
    want = formula(vals, table, q.cpu().numpy(), cu, lens, 128 ** -0.5)
    assert np.abs(got[:cu[1]].double().cpu().numpy() - want[:cu[1]]).max() < 1e-4
    # a chunk longer than max_q_len, and a length over max_seq_len
    if max(qlens) > 1:
        got = run(cache, table, q, cu, lens, torch.float32, max_q=25)
        assert K.kvq_cache_read_errors(cache) == 0x100 and (got[20:] == 7.0).all()
    run(cache, table, q, cu, lens, torch.float32, max_n=95)
    assert K.kvq_cache_read_errors(cache) == 0x8


@pytest.mark.gpu
def test_refusals():
    K = kvq()
    cache, table, _ = build("int8_per_token_head", "f16", 2, 128, [40, 50])
    ints = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    q = torch.randn(20, 4, 128, device="cuda").half()
    out = guarded((20, 4, 128), torch.float16, fill=7.0, name="out")
    ok = dict(q=q, cu_q_lens=ints([0, 10, 20]), block_table=ints(table), seq_lens=ints([40, 50]), out=out, max_q_len=10,
              max_seq_len=50, workspace=torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))
    for change, err in [(dict(q=q.float()), ValueError), (dict(q=q.transpose(0, 1)), ValueError),
                        (dict(cu_q_lens=ints([0, 20])), ValueError), (dict(cu_q_lens=ints([0, 10, 20]).long()), ValueError),
                        (dict(out=out[:19]), ValueError), (dict(prefix_lens=ints([1])), ValueError),
                        (dict(alibi_slopes=torch.ones(3, device="cuda")), ValueError),
                        (dict(window=-1), K.KVQError), (dict(logit_cap=-1.0), K.KVQError),
                        (dict(logit_cap=float("nan")), K.KVQError), (dict(softmax_scale=0.0), K.KVQError),
                        (dict(max_seq_len=10 ** 6), K.KVQError), (dict(max_q_len=-1), K.KVQError),
                        (dict(max_q_len=0), K.KVQError),
                        (dict(mode="nvfp4"), K.KVQError),
                        (dict(q=torch.zeros(20, 3, 128, device="cuda").half(), out=torch.zeros(20, 3, 128, device="cuda")), K.KVQError),
                        (dict(q=torch.zeros(20, 18, 128, device="cuda").half(), out=torch.zeros(20, 18, 128, device="cuda")), K.KVQError)]:
        with pytest.raises(err):
            K.kvq_chunk_attention(cache, **{**ok, **change})
    ns, _, wsb = K.kvq_chunk_plan(cache, 20, 2, 4, max_q_len=10, max_seq_len=50)
    if wsb:
        with pytest.raises(K.KVQError) as e:
            K.kvq_chunk_attention(cache, **{**ok, "workspace": None})
        assert e.value.status == 4
    kcfg = K.make_config(1, 128, 2, 128, "kvarn_k4v2_g128", torch.float16)
    kc = K.kvq_cache_alloc(kcfg, torch.zeros(K.kvq_cache_bytes(kcfg), dtype=torch.uint8, device="cuda"))
    with pytest.raises(K.KVQError) as e:
        K.kvq_chunk_attention(kc, **ok)
    assert e.value.status == 2
    torch.cuda.synchronize()
    assert (out == 7.0).all()
    K.kvq_chunk_attention(cache, **{**ok, "q": q[:0], "out": out[:0]})  # nothing to do
    assert K.kvq_cache_read_errors(cache) == 0


# ---------------------------------------------------------------- as it is used
@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["nvfp4", "int8_per_token_head", "fp8_per_tensor"])
def test_serving_run(mode):
    """A prompt in two chunks and three single tokens through norm + rotation + write and attention, captured and
    replayed on a stream of its own, against the same run without a graph and against the formula over what the
    cache reads back as."""
    K = kvq()
    H, G, D, n = 2, 4, 128, 150
    rng = np.random.default_rng(4)
    cfg = K.make_config(12, 16, H, D, mode, torch.float16)
    pool = guarded(K.kvq_cache_bytes(cfg), torch.uint8, fill=0xFF, name="pool")
    cache = K.kvq_cache_alloc(cfg, pool)
    if mode in TENSOR_SCALED:
        K.kvq_cache_set_tensor_scales(cache, 0.02, 0.002 if mode == "nvfp4" else 0.01)
    table = rng.permutation(12)[:10].astype(np.int32)[None]
    qkv = torch.from_numpy(rng.standard_normal((n, (G * H + 2 * H) * D))).half().cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.from_numpy((table[0, np.arange(n) // 16] * 16 + np.arange(n) % 16).astype(np.int32)).cuda()
    ang = np.arange(n)[:, None] * 1e4 ** (-np.arange(64) / 64)
    tab = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float().cuda()
    w = torch.ones(D, dtype=torch.float16, device="cuda")
    steps = [(0, 83), (83, 147), (147, 148), (148, 149), (149, 150)]
    out, rot = (torch.zeros(n, G * H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    tb = torch.from_numpy(table).cuda()
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dev = [(ints(0, b - a), ints(b)) for a, b in steps]
    wss = [torch.empty(max(16, K.kvq_chunk_plan(cache, b - a, 1, G * H, max_q_len=b - a, max_seq_len=b)[2]),
                       dtype=torch.uint8, device="cuda") for a, b in steps]

    def serve():
        for (a, b), (cu, ln), ws in zip(steps, dev, wss):
            q, k, v = (x.unflatten(1, (-1, D)) for x in qkv[a:b].split([G * H * D, H * D, H * D], 1))
            K.kvq_norm_rope_write(cache, q, k, v, pos[a:b], tab, rot[a:b], slot_mapping=slots[a:b], q_weight=w, k_weight=w)
            K.kvq_chunk_attention(cache, rot[a:b], cu, tb, ln, out[a:b], max_q_len=b - a, max_seq_len=b, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serve()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        serve()
    qkv.copy_(qkv.flip(0) * 0.7)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    out.zero_()
    serve()
    torch.cuda.synchronize()
    assert torch.equal(out, replayed)
    assert K.kvq_cache_read_errors(cache) == 0
    kr, vr = (torch.empty(n, H, D, dtype=torch.float32, device="cuda") for _ in range(2))
    K.kvq_cache_read(cache, slots, kr, vr)
    vals = np.zeros((2, 12, 16, H, D))
    for x, y in zip(vals, (kr, vr)):
        x.reshape(12 * 16, H, D)[slots.cpu().numpy()] = y.double().cpu().numpy()
    want = formula(vals, table, rot.cpu().numpy(), [0, n], [n], D ** -0.5)
    tol = tolerance(want, np.abs(vals[1]).max(), 12.0 * 1.4427 * 4, n, torch.float16, False)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.gpu
def test_one_query_agrees_with_decode():
    K = kvq()
    lens = [33, 400, 1]
    cache, table, _ = build("nvfp4", "f16", 2, 128, lens)
    q = torch.randn(3, 16, 128, device="cuda").half()
    ints = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    got = run(cache, table, q, [0, 1, 2, 3], lens, torch.float32)
    ref = torch.empty(3, 16, 128, device="cuda")
    _, _, wsb = K.kvq_decode_plan(cache, 3, 16, 400)
    K.kvq_decode_attention(cache, q, ints(table), ints(lens), ref, max_seq_len=400,
                           workspace=torch.empty(max(wsb, 16), dtype=torch.uint8, device="cuda"))
    assert (got - ref).abs().max().item() < 1e-4
    assert ctypes.sizeof(K.AttentionOptions) == 24


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ROWS)
@pytest.mark.parametrize("qlens,lens,heads", [([700], [700], (1, 4)), ([300, 64, 90], [1500, 64, 91], (2, 2)),
                                              ([16, 3, 16], [1200, 900, 16], (1, 8))])
def test_longer_chunks(mode, qlens, lens, heads):
    check(mode, "f16", "f16", heads[0], heads[1], 128, qlens, lens)
    check(mode, "f16", "f16", heads[0], heads[1], 128, qlens, lens, cap=3.0, alibi=True, window=200)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f16", "f32"])
@pytest.mark.parametrize("qlens,lens", [([40, 3], [700, 500]), ([200, 9], [900, 40]), ([1, 1], [700, 33])])
def test_pages_below_the_window_are_not_read(io, qlens, lens):
    """A server may give up the pages that no window reaches: their table entries can be anything."""
    K = kvq()
    window = 100
    cache, table, vals = build("fp8_per_token_head", io, 2, 128, lens)
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    q = torch.randn(cu[-1], 8, 128, device="cuda").to(torch.float16 if io == "f16" else torch.float32)
    want = formula(vals, table, q.cpu().numpy(), cu, lens, 128 ** -0.5, window=window)
    for b, (m, n) in enumerate(zip(qlens, lens)):
        table[b, :max(0, n - m - window + 1) // 16] = -7
    got = run(cache, table, q, cu, lens, torch.float32, window=window)
    half = run(cache, table, q, cu, lens, torch.float16, window=window) if io == "f16" else got
    assert K.kvq_cache_read_errors(cache) == 0
    assert np.abs(got.double().cpu().numpy() - want).max() < 1e-4
    assert np.abs(half.double().cpu().numpy() - want).max() < 1e-2


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("qlens,lens", [([40, 3], [300, 50]), ([300], [900])])
def test_nan_query_and_nan_in_unseen_keys(qlens, lens, out):
    """A NaN query makes its own row NaN and no other; NaN keys after a query's position do not reach it."""
    K = kvq()
    cache, table, vals = build("int8_per_token_head", "f16", 1, 128, lens)
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    q = torch.randn(cu[-1], 4, 128, device="cuda").half()
    want = formula(vals, table, q.cpu().numpy(), cu, lens, 128 ** -0.5)
    q[1, 2, 5] = float("nan")
    # the key scale of the first sequence's last token
    tok = lens[0] - 1
    blk = cache.pool[256:].view(cache.cfg.num_pages, -1)[int(table[0, tok // 16])]
    blk[4096:4096 + 64].view(torch.float32)[tok % 16] = float("nan")
    got = run(cache, table, q, cu, lens, torch.float16 if out == "f16" else torch.float32).double().cpu().numpy()
    last = qlens[0] - 1
    assert np.isnan(got[1, 2]).all() and np.isnan(got[last]).all()
    keep = np.ones(got.shape[:2], bool)
    keep[1, 2] = keep[last] = False
    assert np.isfinite(got[keep]).all() and np.abs(got[keep] - want[keep]).max() < 5e-3


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int8_per_token_head", "nvfp4", "fp8_per_tensor"])
@pytest.mark.parametrize("cap", [0.25, 4.0, 400.0])
def test_scores_far_past_the_cap(mode, cap):
    """Scores of about 11 in size, so that tanh is taken from its linear part to far past where it is 1."""
    check(mode, "f16", "f16", 1, 8, 128, [70, 1, 20], [70, 260, 301], cap=cap, scale=1.0)
    check(mode, "f16", "f32", 2, 2, 128, [150, 3], [150, 700], cap=cap, scale=1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_nan_with_a_cap(out):
    """With capped scores too a NaN stays in its row, and unseen NaN keys reach none."""
    K = kvq()
    qlens, lens = [300, 5], [300, 400]
    cache, table, vals = build("int8_per_token_head", "f16", 1, 128, lens)
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    q = torch.randn(cu[-1], 4, 128, device="cuda").half()
    want = formula(vals, table, q.cpu().numpy(), cu, lens, 128 ** -0.5, cap=3.0)
    q[1, 2, 5] = float("nan")
    tok = lens[0] - 1
    blk = cache.pool[256:].view(cache.cfg.num_pages, -1)[int(table[0, tok // 16])]
    blk[4096:4096 + 64].view(torch.float32)[tok % 16] = float("nan")
    got = run(cache, table, q, cu, lens, torch.float16 if out == "f16" else torch.float32,
              logit_cap=3.0).double().cpu().numpy()
    last = qlens[0] - 1
    assert np.isnan(got[1, 2]).all() and np.isnan(got[last]).all()
    keep = np.ones(got.shape[:2], bool)
    keep[1, 2] = keep[last] = False
    assert np.isfinite(got[keep]).all() and np.abs(got[keep] - want[keep]).max() < 5e-3


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f16", "f32"])
@pytest.mark.parametrize("cap", [1.0e-10, 1024.0])
def test_the_smallest_and_the_largest_cap(io, cap):
    check("int8_per_token_head", io, io, 1, 8, 128, [70, 1, 20], [70, 260, 301], cap=cap)
    check("int8_per_token_head", io, io, 2, 4, 128, [1, 1], [300, 17], cap=cap)
    check("nvfp4", io, io, 2, 1, 32, [70, 3], [70, 90], cap=cap)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [1.0e-11, 1025.0, 3.0e38, float("inf"), -0.5])
def test_caps_out_of_range_are_refused(cap):
    K = kvq()
    cache, table, _ = build("nvfp4", "f16", 1, 128, [20])
    q = torch.zeros(4, 8, 128, device="cuda", dtype=torch.float16)
    with pytest.raises(K.KVQError):
        run(cache, table, q, np.array([0, 4], np.int32), [20], torch.float16, logit_cap=cap)


@pytest.mark.gpu
def test_a_scale_too_large_for_the_cap_is_refused():
    """The kernels work with softmax_scale / logit_cap."""
    K = kvq()
    cache, table, _ = build("nvfp4", "f16", 1, 128, [20])
    q = torch.zeros(4, 8, 128, device="cuda", dtype=torch.float16)
    with pytest.raises(K.KVQError):
        run(cache, table, q, np.array([0, 4], np.int32), [20], torch.float16, logit_cap=1.0e-10, softmax_scale=1.0e30)


@pytest.mark.gpu
@pytest.mark.parametrize("qlens,lens", [([300, 5], [300, 400]), ([1, 1], [700, 20]), ([1, 1], [20000, 33]),
                                        ([1] * 40, [90] * 40)])
def test_a_nan_stays_in_its_row_under_a_large_cap(qlens, lens):
    """A NaN query beside heads with small scores and with scores past the cap, in a chunk and in a single token."""
    K = kvq()
    cache, table, vals = build("int8_per_token_head", "f16", 1, 128, lens)
    cu = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    q = torch.randn(cu[-1], 4, 128, device="cuda").half()
    q[0, 1] *= 3000.0
    cap = 1000.0
    want = formula(vals, table, q.cpu().numpy(), cu, lens, 128 ** -0.5, cap=cap)
    q[0, 2, 5] = float("nan")
    got = run(cache, table, q, cu, lens, torch.float16, logit_cap=cap).double().cpu().numpy()
    assert np.isnan(got[0, 2]).all()
    keep = np.ones(got.shape[:2], bool)
    keep[0, 1:3] = False
    tol = tolerance(want, np.abs(vals[1][np.isfinite(vals[1])]).max(), 1.4427 * cap, max(lens), torch.float16, False)
    assert np.isfinite(got[0, 1]).all() and (np.abs(got - want) <= tol)[keep].all()

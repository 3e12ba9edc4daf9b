"""kvq_chunk_attention where its softmax reference and its weights have to be right:
scores that jump inside a tile, and value scales far apart.  Every row is held to
the values that it sees itself."""
import numpy as np
import pytest
import torch

from _helpers import header_scales, kvq
from test_chunk_attention import build, run
from test_norm_rope_read import pool_values


def store(cache, table, b, k, v):
    """Write k, v [n][H][D] (numpy) as sequence b of `table`; the pool's values afterwards."""
    n = len(k)
    t = np.arange(n)
    slots = torch.from_numpy((table[b, t // 16] * 16 + t % 16).astype(np.int32)).cuda()
    kvq().kvq_quantize_write(cache, *(torch.from_numpy(x).to(cache.io_dtype).cuda() for x in (k, v)), slots)


def values(cache, mode):
    torch.cuda.synchronize()
    return pool_values(mode, cache.pool.cpu().numpy(), cache.cfg.num_pages, cache.heads, cache.head_dim,
                       *header_scales(cache))


def exact_rows(vals, table, q, cu, lens, scale, window=0, cap=0.0, weight=2.0 ** -20, slopes=None, prefix=None):
    """The formula in 64 bits and, for every output, a bound on its error.

    A score is an fp32 sum of D products (the products are exact: codes of at most 9 bits times fp16, or times the
    halves of an fp32 value), in steps of 16: 16 roundings (2^-23 where sums are cut off) of sum |q k|, four more of the
    score itself.  A weight is within that, the exponential (2^-22) and its own bits (`weight`: both), or within half
    of fp16's smallest step, 2^-25, where the row's largest is held at 2^2 at least: 2^-27 of weight x value; the sums over n tokens take n / 16 + 16 steps."""
    H, (Hq, D) = vals.shape[3], q.shape[1:]
    want, tol = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for b, n in enumerate(lens):
        t = np.arange(n)
        k, v = vals[:, table[b, t // 16], t % 16]
        m = cu[b + 1] - cu[b]
        for i in range(m):
            p = n - m + i
            see = ((t <= p) & ((t > p - window) if window else True)) | (t < (0 if prefix is None else prefix[b]))
            for h in range(Hq):
                x = q[cu[b] + i, h].astype(np.float64)
                kk, vv = k[see, h // (Hq // H)], v[see, h // (Hq // H)]
                s = scale * (kk @ x)
                ds = 16 * 2.0 ** -23 * scale * (np.abs(kk) @ np.abs(x)) + 8 * 2.0 ** -23 * np.abs(s) + 2.0 ** -21
                if cap:
                    s = cap * np.tanh(s / cap)
                    ds = ds + 2.0 ** -22 * cap
                if slopes is not None:
                    far = float(slopes[h]) * np.abs(p - t[see])
                    s, ds = s - far, ds + 4 * 2.0 ** -23 * far
                w = np.exp(s - s.max())
                w /= w.sum()
                want[cu[b] + i, h] = w @ vv
                ds = ds + weight + (see.sum() / 16 + 16) * 2.0 ** -23
                mag = w @ np.abs(vv)  # of every channel
                tol[cu[b] + i, h] = (w * ds) @ np.abs(vv) + (w @ ds) * mag + \
                    see.sum() * 2.0 ** -27 * (w * np.abs(vv).max(1)).max()
    return want, tol


def hold(got, want, tol):
    dt = got.dtype
    got = got.double().cpu().numpy()
    # its own rounding: eps / 2 of the value, half a step of the smallest numbers
    tol = tol + torch.finfo(dt).eps / 2 * np.abs(want) + (2.0 ** -25 if dt == torch.float16 else 0.0)
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"worst {np.max(err / tol):.3g} of the tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int8_per_token_head", "fp8_per_tensor", "nvfp4"])
@pytest.mark.parametrize("m,G", [(150, 2), (9, 8)])
def test_scores_that_jump_twice_in_a_tile(mode, m, G):
    """Tiles behind the first whose scores rise by 2^20 and more in their first 64 tokens and again in the other 64,
    rows of one warp in different halves: O is rescaled twice within one tile."""
    D, n = 128, 128 * 5 + 40
    cache, table, _ = build(mode, "f16", 1, D, [n])
    rng = np.random.default_rng(3)
    k = rng.standard_normal((n, 1, D)) * 0.05
    v = rng.standard_normal((n, 1, D))
    tile, half = np.arange(n) // 128, np.arange(n) // 64 % 2
    rise = 4 - tile  # the tiles are met from the last to the first
    k[:, 0, 0] += 1.0 * rise + 0.5 * half      # both halves
    k[:, 0, 1] += 1.0 * rise * (half == 0)     # the first half alone
    k[:, 0, 2] += 1.0 * rise * (half == 1)     # the second half alone
    kvq().kvq_cache_set_tensor_scales(cache, 6.0 / (448 if mode == "fp8_per_tensor" else 2688), 5.0 / 2688)
    store(cache, table, 0, k, v)
    vals = values(cache, mode)
    q = rng.standard_normal((m, G, D)) * 0.3
    for r in range(m * G):
        q[r // G, r % G, r % 3] += 300.0  # times 1 / sqrt(128) and log2 e: 38 a step
    q = torch.from_numpy(q).half().cuda()
    got = run(cache, table, q, [0, m], [n], torch.float16)
    assert kvq().kvq_cache_read_errors(cache) == 0
    hold(got, *exact_rows(vals, table, q.cpu().numpy(), [0, m], [n], D ** -0.5))


def batch(mode, io, out, H, G, D, qlens, lens, shape_v, q_gain=1.0, k_gain=1.0, sink=False, window=0, seed=7):
    """Sequences whose values are standard normal times shape_v(n) (a factor per token) against the formula; with
    `sink` the first token takes most of every row's weight."""
    cache, table, _ = build(mode, io, H, D, lens)
    rng = np.random.default_rng(seed)
    for b, n in enumerate(lens):
        k = rng.standard_normal((n, H, D))
        if sink:
            k[0] = 0.9 * np.sqrt(D)  # against queries with a mean of 0.15 sqrt(128 / D): a score of about 17
        store(cache, table, b, k * k_gain, rng.standard_normal((n, H, D)) * shape_v(n)[:, None, None])
    vals = values(cache, mode)
    cu = np.concatenate([[0], np.cumsum(qlens)])
    dt, odt = (torch.float16 if x == "f16" else torch.float32 for x in (io, out))
    q = rng.standard_normal((cu[-1], H * G, D)) + (0.15 * np.sqrt(128 / D) if sink else 0.0)
    q = torch.from_numpy(q * q_gain).to(dt).cuda()
    scale = D ** -0.5 / (q_gain * k_gain)
    got = run(cache, table, q, cu, lens, odt, softmax_scale=scale, window=window)
    assert kvq().kvq_cache_read_errors(cache) == 0
    hold(got, *exact_rows(vals, table, q.cpu().numpy(), cu, lens, float(np.float32(scale)), window))


CHUNK = ([70, 9], [330, 60])
PROMPT = ([300], [300])  # more than 128 rows
SINGLE = ([1, 1, 1], [1, 300, 1500])
PT = ["int8_per_token_head", "fp8_per_token_head", "int4_per_token_head"]


@pytest.mark.gpu
@pytest.mark.parametrize("mode", PT + ["fp8_per_tensor", "nvfp4"])
@pytest.mark.parametrize("lens", [CHUNK, PROMPT], ids=["chunk", "prompt"])
def test_weights_keep_their_bits(mode, lens):
    """fp16 outputs are their exact values rounded, give or take 2^-20 of the weights."""
    batch(mode, "f16", "f16", 1, 2, 128, *lens, lambda n: np.full(n, 0.4))


# values by token: a factor that falls, grows or scatters by orders of magnitude
SHAPES = {
    "small sink": lambda n: np.where(np.arange(n) == 0, 2.0 ** -14, 1.0),
    "tiny sink": lambda n: np.where(np.arange(n) == 0, 2.0 ** -22, 1.0),
    "scattered": lambda n: 10.0 ** (6.0 * np.random.default_rng(n).random(n) - 4.0),
    "last one large": lambda n: np.where(np.arange(n) == n - 1, 6e3, 1e-2),
}
FAR = {"last one huge": lambda n: np.where(np.arange(n) == n - 1, 1e6, 1e-2),
       "growing": lambda n: 10.0 ** np.linspace(-8.0, 8.0, n)}


@pytest.mark.gpu
@pytest.mark.parametrize("mode", PT)
@pytest.mark.parametrize("io,out,D,shape", [(io, out, D, x) for io, out, D in (("f32", "f32", 128), ("f32", "f32", 32), ("f16", "f32", 128), ("f16", "f16", 32))
                                            for x in (*SHAPES, *(FAR if io == "f32" else ()))])  # (FAR lies outside fp16)
def test_value_scales_far_apart_mma(mode, io, out, D, shape):
    """Heavy tokens with small values, and large values that most rows do not see."""
    batch(mode, io, out, 1, 2, D, *CHUNK, {**SHAPES, **FAR}[shape], sink="sink" in shape)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", PT)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("lens", [CHUNK, PROMPT], ids=["chunk", "prompt"])
def test_value_scales_far_apart_fp16(mode, lens, shape):
    batch(mode, "f16", "f16", 1, 2, 128, *lens, SHAPES[shape], sink="sink" in shape)


@pytest.mark.gpu
@pytest.mark.parametrize("io,out,lens", [("f32", "f32", CHUNK), ("f16", "f16", CHUNK), ("f16", "f16", PROMPT), ("f16", "f16", SINGLE),
                                         ("f32", "f32", SINGLE)])
def test_large_values_below_the_window(io, out, lens):
    batch("int8_per_token_head", io, out, 1, 4, 128, *lens, lambda n: np.where(np.arange(n) % 48 < 8, 6e3, 1e-2), window=20)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", PT)
@pytest.mark.parametrize("io,out,D,size", [(io, out, D, x) for io, out, D in (("f32", "f32", 128), ("f32", "f32", 32), ("f16", "f32", 128), ("f16", "f16", 128))
                                           for x in (1e-12, 1e-4, 1e-2, 1.0, 3e3, 1e7, 1e30) if io == "f32" or 1e-5 < x < 1e4])
def test_single_tokens_values_of_any_size(mode, io, out, D, size):
    batch(mode, io, out, 2, 2, D, *SINGLE, lambda n: np.full(n, size))


@pytest.mark.gpu
@pytest.mark.parametrize("mode", PT)
@pytest.mark.parametrize("io,shape", [("f16", x) for x in SHAPES] + [("f32", x) for x in (*SHAPES, *FAR)])
def test_single_tokens_value_scales_far_apart(mode, io, shape):
    batch(mode, io, "f32", 1, 4, 128, *SINGLE, {**SHAPES, **FAR}[shape], sink="sink" in shape)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int8_per_token_head", "fp8_per_token_head", "int4_per_token_head"])
@pytest.mark.parametrize("D", [32, 128])
@pytest.mark.parametrize("lens", [CHUNK, SINGLE], ids=["chunk", "single"])
@pytest.mark.parametrize("size", [1e-12, 1e-5, 1e5, 1e12])
def test_fp32_queries_of_any_size(mode, D, lens, size):
    batch(mode, "f32", "f32", 2, 2, D, *lens, lambda n: np.ones(n), q_gain=size, k_gain=1.0 / size)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["fp8_per_tensor", "nvfp4"])
@pytest.mark.parametrize("qlens,lens", [([300, 40], [900, 40]), ([1, 1], [500, 3])])
def test_a_score_factor_that_underflows(mode, qlens, lens):
    """softmax_scale times the keys' tensor scale below fp32: all scores 0, each row the mean of the values that it sees."""
    cache, table, _ = build(mode, "f16", 1, 128, lens)
    ks, vs = header_scales(cache)
    kvq().kvq_cache_set_tensor_scales(cache, 1e-30, vs)
    vals = values(cache, mode)
    cu = np.concatenate([[0], np.cumsum(qlens)])
    q = torch.from_numpy(np.random.default_rng(2).standard_normal((cu[-1], 2, 128))).half().cuda()
    got = run(cache, table, q, cu, lens, torch.float32, softmax_scale=1e-30)
    hold(got, *exact_rows(vals, table, q.cpu().numpy(), cu, lens, 1e-30))


@pytest.mark.gpu
@pytest.mark.parametrize("mode", PT)
@pytest.mark.parametrize("io,lens", [("f16", CHUNK), ("f16", PROMPT), ("f16", SINGLE), ("f32", CHUNK), ("f32", SINGLE)])
@pytest.mark.parametrize("cap,window,alibi,pre", [(4.0, 0, False, False), (0.0, 0, True, False), (0.0, 40, False, True), (4.0, 40, True, True)])
def test_options_with_scattered_values(mode, io, lens, cap, window, alibi, pre):
    """Caps, biases, windows and prefixes over values six orders of magnitude apart and slots of zero scale."""
    qlens, lens = lens
    cache, table, _ = build(mode, io, 1, 128, lens)
    cache.pool[256:].zero_()
    rng = np.random.default_rng(5)
    for b, n in enumerate(lens):
        k, v = rng.standard_normal((2, n, 1, 128))
        v *= SHAPES["scattered"](n)[:, None, None]
        keep = np.arange(n) % 29 != 28  # the others' slots stay zero: zero scores, zero values
        t = np.arange(n)[keep]
        slots = torch.from_numpy((table[b, t // 16] * 16 + t % 16).astype(np.int32)).cuda()
        kvq().kvq_quantize_write(cache, *(torch.from_numpy(x[keep]).to(cache.io_dtype).cuda() for x in (k, v)), slots)
    vals = values(cache, mode)
    cu = np.concatenate([[0], np.cumsum(qlens)])
    q = torch.from_numpy(rng.standard_normal((cu[-1], 2, 128))).to(cache.io_dtype).cuda()
    slopes = np.array([0.25, 2.0 ** -6], np.float32) if alibi else None
    prefix = np.array([n // 3 for n in lens], np.int32) if pre else None
    got = run(cache, table, q, cu, lens, torch.float32, logit_cap=cap, window=window,
              alibi_slopes=None if slopes is None else torch.from_numpy(slopes).cuda(),
              prefix_lens=None if prefix is None else torch.from_numpy(prefix).cuda())
    assert kvq().kvq_cache_read_errors(cache) == 0
    hold(got, *exact_rows(vals, table, q.cpu().numpy(), cu, lens, 128 ** -0.5, window, cap, slopes=slopes, prefix=prefix))


@pytest.mark.gpu
@pytest.mark.parametrize("H,G,qlens,n", [(1, 8, [8] * 100, 4000), (2, 3, [40] * 7, 900), (8, 4, [700], 700), (1, 1, [300, 2], 9000)])
def test_the_workspace_serves_both_output_types(H, G, qlens, n):
    """fp32 outputs of fp16 queries take the kernel that fp32 queries take, in as many parts, so they need as much."""
    K = kvq()
    need = []
    for dt in (torch.float16, torch.float32):
        cfg = K.make_config(1, 16, H, 128, "int8_per_token_head", dt)
        cache = K.kvq_cache_alloc(cfg, torch.zeros(K.kvq_cache_bytes(cfg), dtype=torch.uint8, device="cuda"))
        need.append(K.kvq_chunk_plan(cache, sum(qlens), len(qlens), H * G, max_q_len=max(qlens), max_seq_len=n)[2])
    assert need[0] >= need[1]
    cache, table, _ = build("int8_per_token_head", "f16", H, 128, [n])
    q = torch.zeros(sum(qlens), H * G, 128, device="cuda", dtype=torch.float16)
    cu = np.concatenate([[0], np.cumsum(qlens)])
    for dt in (torch.float16, torch.float32):  # (guarded workspaces of just the planned size)
        run(cache, np.repeat(table, len(qlens), 0), q, cu, [n] * len(qlens), dt)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int8_per_token_head", "fp8_per_tensor"])
@pytest.mark.parametrize("io,D,m", [("f16", 128, 40), ("f32", 128, 40), ("f32", 32, 40)])
def test_sums_over_many_tokens(mode, io, D, m):
    """fp32 means over 20000 values near 1: at most 256 of a row's additions in a row are cut off, by 2^-23 of a sum that
    grows evenly, which makes 128 x 2^-23; weights and the other additions are within 2^-18."""
    H, B, n = 8, 20, 20000  # enough rows that a range is not split much; all sequences read the same pages
    K = kvq()
    cache, table, _ = build(mode, io, H, D, [n])
    K.kvq_cache_set_tensor_scales(cache, 1.0, 2.0 / 448)
    v = 1.0 + 0.1 * np.random.default_rng(1).standard_normal((n, H, D))
    store(cache, table, 0, np.zeros((n, H, D)), v)
    vals = values(cache, mode)[1][table[0, np.arange(n) // 16], np.arange(n) % 16]
    q = torch.randn(B * m, 2 * H, D, device="cuda").to(cache.io_dtype)
    got = run(cache, np.repeat(table, B, 0), q, np.arange(0, B * m + 1, m), [n] * B, torch.float32)
    want = (np.cumsum(vals, 0) / np.arange(1, n + 1)[:, None, None])[n - m:]
    err = np.abs(got.double().cpu().numpy().reshape(B, m, H, 2, D) - want[None, :, :, None]) / want[None, :, :, None]
    assert err.max() <= 128 * 2.0 ** -23 + 2.0 ** -18, f"{err.max():.3g}"

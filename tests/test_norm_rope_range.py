"""kvq_norm_rope_write on rows with infinities and NaN, and on fp32 rows whose
squares leave fp32's range."""
import numpy as np
import pytest
import torch

from _helpers import guarded, kvq


def formula(x, w, ang, rot, interleaved, eps):
    """In 64 bits, by IEEE rules for infinities and NaN; values that are not rotated enter no product."""
    with np.errstate(all="ignore"):
        y = x.astype(np.float64)
        if w is not None:
            y = y * w.astype(np.float64) / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps)))
        z = y.copy()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = ang[:, i].astype(np.float64)[:, None], ang[:, rot // 2 + i].astype(np.float64)[:, None]
            z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    return z


def rotate(x, w, pos, tab, rot, interleaved, eps):
    """Queries x [T][Hq][D] through the call."""
    K = kvq()
    T, Hq, D = x.shape
    cfg = K.make_config(1, 16, 1, D, "int8_per_token_head", torch.float16 if x.dtype == np.float16 else torch.float32)
    cache = K.kvq_cache_alloc(cfg, guarded(K.kvq_cache_bytes(cfg), torch.uint8, fill=0, name="pool"))
    q = torch.from_numpy(x).cuda()
    out = guarded((T, Hq, D), q.dtype, fill=5.0, name="q_out")
    kw = dict(q_weight=None if w is None else torch.from_numpy(w).cuda(), eps=eps, interleaved=interleaved)
    args = (torch.from_numpy(pos).cuda(), torch.from_numpy(tab).cuda()) if rot else (None, None)
    K.kvq_norm_rope_write(cache, q, torch.zeros(T, 1, D, dtype=q.dtype, device="cuda"), None, *args, out, **kw)
    torch.cuda.synchronize()
    return out.cpu().numpy()


def table(rot):
    ang = np.arange(50)[:, None] * 100.0 ** (-np.arange(max(rot // 2, 1)) / max(rot // 2, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("io", [np.float16, np.float32])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 64, False), (128, 64, True), (128, 0, False),
                                               (32, 32, True), (32, 16, False)])
@pytest.mark.parametrize("norm", [False, True])
def test_infinities_and_nan(io, D, rot, interleaved, norm):
    """One, and two, values of a row are not finite, in the rotated part and behind it."""
    rng = np.random.default_rng(D + rot)
    T, Hq = 40, 3
    x = rng.standard_normal((T, Hq, D)).astype(io)
    for t in range(T):
        for h in range(Hq):
            x[t, h, (7 * t + 5 * h) % D] = (np.inf, -np.inf, np.nan)[(t + h) % 3]
            if t % 2:
                x[t, h, (7 * t + 5 * h + D // 2) % D] = np.inf
    w = (1.0 + 0.2 * rng.standard_normal(D)).astype(io) if norm else None
    tab = table(rot)
    pos = rng.integers(1, 50, T).astype(np.int32)
    got = rotate(x, w, pos, tab, rot, interleaved, 1e-6)
    z = formula(x, w, tab[pos], rot, interleaved, 1e-6)
    with np.errstate(all="ignore"):
        want = z.astype(io)
        near = ((z * (1 - 2.0 ** -40)).astype(io) != (z * (1 + 2.0 ** -40)).astype(io)) & np.isfinite(z)
    same = (got == want) | (np.isnan(got) & np.isnan(want)) | near
    assert same.all(), f"{(~same).sum()} of {same.size} values differ from the formula"


@pytest.mark.gpu
@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (0, False)])
@pytest.mark.parametrize("size", [2.0 ** -125, 2.0 ** -110, 2.0 ** -70, 1e-12, 1e12, 2.0 ** 70, 2.0 ** 110])
def test_fp32_rows_of_any_size(rot, interleaved, size):
    """The squares of 2^+-70 leave fp32's range; the normed rows are of size 1."""
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((9, 2, 128)) * size).astype(np.float32)
    x[4, 1] = 0.0  # with eps 0: 0 / 0
    w = (1.0 + 0.2 * rng.standard_normal(128)).astype(np.float32)
    tab = table(rot)
    pos = rng.integers(0, 50, 9).astype(np.int32)
    for eps in (1e-6, 1e-30, 0.0):
        got = rotate(x, w, pos, tab, rot, interleaved, eps)
        z = formula(x, w, tab[pos], rot, interleaved, eps)
        assert np.isnan(got[4, 1]).all() if eps == 0.0 else (got[4, 1] == 0.0).all()
        got[4, 1] = z[4, 1] = 0.0
        near = (z * (1 - 2.0 ** -40)).astype(np.float32) != (z * (1 + 2.0 ** -40)).astype(np.float32)
        normal = (np.abs(z) > 2.0 ** -90) | (z == 0)  # below it the low words of the products leave fp32
        bad = (got != z.astype(np.float32)) & ~near & normal
        assert not bad.any(), f"{bad.sum()} values are not the rounded formula"
        # the smallest step, 2^-149, of x w and of the rotated value, times 1 / sqrt(eps) = 2^10 where nothing is scaled
        assert (np.abs(got - z) <= 2.0 ** -22 * np.abs(z) + 4 * 2.0 ** -139).all()

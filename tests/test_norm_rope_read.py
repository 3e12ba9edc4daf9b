"""kvq_cache_read and kvq_norm_rope_write: values against the pool layout and
the formulas in 64 bits, the written pool bit for bit against a write of the
correctly rounded keys, refusals, and the two together."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from _helpers import MODE_NAMES, TENSOR_SCALED, guarded, kvq

ROWS = [m for m in MODE_NAMES if not m.startswith("kvarn")]


# ---------------------------------------------------------------- a small cache
def hadamard(n):
    h = np.ones((1, 1))
    while len(h) < n:
        h = np.block([[h, h], [h, -h]])
    return h / np.sqrt(n)


def e4m3(b):
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    mag = np.where(e == 0, m * 2.0 ** -9, (8.0 + m) * np.exp2(e - 10.0))
    return np.where(b >> 7 == 1, -mag, mag)


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def pool_values(mode, pool, num_pages, H, D, ks, vs):
    """[2][pages][P][H][D] in 64 bits, from the layout text of kvq.h."""
    P = 128 if mode.startswith("kvarn") else 16
    blk = pool[256:].reshape(num_pages * H, -1)
    out = np.zeros((2, num_pages, P, H, D))
    for i in range(num_pages * H):
        b = blk[i]
        f32 = lambda a, n: b[a:a + 4 * n].view(np.float32).astype(np.float64)  # noqa: E731
        for side in (0, 1):
            st = float(np.float32((ks, vs)[side]))
            if mode.startswith("kvarn"):
                m = P * D * 3 // 4
                if side == 0:
                    by = b[:P * D // 2].reshape(P, D // 2)
                    c = np.stack([by & 15, by >> 4], -1).reshape(P, D)
                    sc, z, cd, r = f32(m, D), f32(m + 4 * D, D), f32(m + 8 * D, D), f32(m + 12 * D, P)
                    y = r[:, None] * cd * (sc * c + z)
                else:
                    m += 4 * (3 * D + P)
                    by = b[P * D // 2:P * D * 3 // 4].reshape(P, D // 4)
                    c = np.stack([(by >> s) & 3 for s in (0, 2, 4, 6)], -1).reshape(P, D)
                    sc, z, r, cd = f32(m, P), f32(m + 4 * P, P), f32(m + 8 * P, P), f32(m + 12 * P, D)
                    y = r[:, None] * cd * (sc[:, None] * c + z[:, None])
                x = y @ hadamard(D)
            elif mode in ("fp8_per_tensor", "fp8_per_token_head", "int8_per_token_head"):
                c = b[side * P * D:(side + 1) * P * D].reshape(P, D)
                x = c.view(np.int8).astype(np.float64) if mode[0] == "i" else e4m3(c)
                x = x * (st if mode == "fp8_per_tensor" else f32(2 * P * D + 4 * P * side, P)[:, None])
            else:
                by = b[side * P * D // 2:(side + 1) * P * D // 2]
                n = np.stack([by & 15, by >> 4], -1).reshape(-1)
                if mode == "int4_per_token_head":
                    if side == 0:
                        n = n.reshape(P, D // 8, 8)[..., [0, 4, 1, 5, 2, 6, 3, 7]].reshape(P, D)
                    else:
                        n = n.reshape(P // 2, D // 4, 2, 4).transpose(0, 2, 1, 3).reshape(P, D)
                    x = np.where(n > 7, n.astype(int) - 16, n) * f32(P * D + 4 * P * side, P)[:, None]
                else:
                    n = n.reshape(P, D) if side == 0 else n.reshape(P // 2, D, 2).transpose(0, 2, 1).reshape(P, D)
                    s = e4m3(b[P * D + side * P * D // 16:P * D + (side + 1) * P * D // 16]).reshape(P, D // 16)
                    x = np.where(n > 7, -1.0, 1.0) * E2M1[n & 7] * np.repeat(s, 16, 1) * st
            out[side, i // H, :, i % H] = x
    return out


def filled(mode, num_pages, H, D, io="f16", seed=3, scale=1.0):
    """A GPU cache written with random tokens in every slot, its pool bytes, tensor scales and the tokens."""
    K = kvq()
    P = 128 if mode.startswith("kvarn") else 16
    dt = torch.float16 if io == "f16" else torch.float32
    cfg = K.make_config(num_pages, P, H, D, mode, dt)
    pool = guarded(K.kvq_cache_bytes(cfg), torch.uint8, fill=0xCD, name="pool")
    cache = K.kvq_cache_alloc(cfg, pool)
    rng = np.random.default_rng(seed)
    k, v = (torch.from_numpy(rng.standard_normal((num_pages * P, H, D)) * scale).to(dt).cuda() for _ in range(2))
    ks = vs = 1.0
    if mode in TENSOR_SCALED:
        ks = vs = float(np.float32(5.0 * scale / (448.0 if mode == "fp8_per_tensor" else 2688.0)))
        K.kvq_cache_set_tensor_scales(cache, ks, vs)
    slots = torch.arange(num_pages * P, dtype=torch.int32, device="cuda")
    K.kvq_quantize_write(cache, k, v, slots)
    torch.cuda.synchronize()
    return cache, pool.cpu().numpy(), ks, vs


# ---------------------------------------------------------------- refusals (CPU)
def test_refusals_before_device_work():
    K = kvq()
    lib = K.lib()
    assert lib.kvq_cache_read(None, None, 1, None, None, 0, None) == 1
    assert lib.kvq_norm_rope_write(None, None, 1, None) == 1
    r = K.NormRope()
    assert lib.kvq_norm_rope_write(None, ctypes.byref(r), 1, None) == 1


# ---------------------------------------------------------------- reading back
@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", ["f16", "f32"])
@pytest.mark.parametrize("mode,H,D", [(m, h, d) for m in ROWS for h, d in ((3, 32), (5, 128))] +
                         [("kvarn_k4v2_g128", 3, 128)])
def test_read_values(mode, H, D, out_dtype):
    K = kvq()
    pages = 3 if mode.startswith("kvarn") else 9
    P = 128 if mode.startswith("kvarn") else 16
    cache, pool, ks, vs = filled(mode, pages, H, D)
    ref = pool_values(mode, pool, pages, H, D, ks, vs).reshape(2, pages * P, H, D)
    dt = torch.float16 if out_dtype == "f16" else torch.float32
    rng = np.random.default_rng(5)
    for n in (1, 2, 37, 301):
        slots = rng.integers(0, pages * P, n).astype(np.int32)  # any order, repeats included
        slots[n // 2] = -1
        slots[-1] = slots[0]
        sd = torch.from_numpy(slots).cuda()
        ko, vo = (guarded((n, H, D), dt, fill=7.0, name="out") for _ in range(2))
        K.kvq_cache_read(cache, sd, ko, vo)
        one = guarded((n, H, D), dt, fill=7.0, name="out")
        K.kvq_cache_read(cache, sd, None, one)
        torch.cuda.synchronize()
        assert torch.equal(one, vo)
        for side, got in ((0, ko), (1, vo)):
            g = got.double().cpu().numpy()
            want = ref[side][np.maximum(slots, 0)]
            want[slots < 0] = 7.0
            # one rounding to the output type (half a step, eps / 2) and at most
            # three fp32 roundings before it; KVarN: a sum of 128 terms in seven
            # levels, each level and each of its five products within 2^-24 of
            # the row's absolute sum, at most sqrt(128) times its norm / sqrt(128)
            eps = torch.finfo(dt).eps / 2
            tol = (eps + 4 * 2.0 ** -24) * np.abs(want) + 2.0 ** -25
            if mode.startswith("kvarn"):
                tol = tol + 12 * 2.0 ** -24 * np.linalg.norm(want, axis=-1, keepdims=True) * 11.4
            assert (np.abs(g - want) <= tol).all()
    assert K.kvq_cache_read_errors(cache) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["int8_per_token_head", "kvarn_k4v2_g128"])
def test_read_flags_slots_past_the_pool(mode):
    K = kvq()
    cache, pool, _, _ = filled(mode, 2, 2, 128)
    P = 128 if mode.startswith("kvarn") else 16
    slots = torch.tensor([0, 2 * P, 1], dtype=torch.int32, device="cuda")
    out = guarded((3, 2, 128), torch.float32, fill=-3.0, name="out")
    K.kvq_cache_read(cache, slots, out, None)
    torch.cuda.synchronize()
    assert (out[1] == -3.0).all() and not (out[[0, 2]] == -3.0).any()
    assert K.kvq_cache_read_errors(cache) == 1
    with pytest.raises(ValueError):
        K.kvq_cache_read(cache, slots.long(), out, None)
    with pytest.raises(ValueError):
        K.kvq_cache_read(cache, slots, out[:, :1], None)
    with pytest.raises(ValueError):
        K.kvq_cache_read(cache, slots, out.transpose(0, 1), None)
    with pytest.raises(ValueError):
        K.kvq_cache_read(cache, slots, None, None)


# ---------------------------------------------------------------- norm + rotation + write
def rotated(x, w, ang, rot, interleaved, eps):
    """The formula in extended precision (x86 and Arm long double differ: fp64 is 2^-53, well below 2^-44)."""
    y = x.astype(np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps))) * w.astype(np.float64)
    z = y.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = ang[:, i].astype(np.float64)[:, None], ang[:, rot // 2 + i].astype(np.float64)[:, None]
        z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    return z


def near_border(z, dt):
    """Values whose rounding to dt the 2^-44 of the kernel's arithmetic (and fp64's own 2^-53 terms) need not settle."""
    r = 2.0 ** -40
    return (z * (1 - r)).astype(dt) != (z * (1 + r)).astype(dt)


CASES = [  # mode, io, Hq, Hkv, D, rot, interleaved, norm, tokens
    ("int8_per_token_head", "f16", 5, 1, 128, 128, False, True, 33),
    ("fp8_per_token_head", "f16", 8, 2, 128, 64, False, True, 1),
    ("fp8_per_tensor", "f16", 4, 4, 32, 32, False, True, 70),
    ("nvfp4", "f16", 14, 2, 128, 128, True, True, 50),
    ("nvfp4_4over6", "f16", 3, 3, 128, 32, False, False, 31),
    ("int4_per_token_head", "f16", 9, 9, 128, 128, False, True, 67),
    ("int4_per_token_head", "f16", 2, 1, 32, 16, True, True, 130),
    ("int8_per_token_head", "f32", 4, 4, 32, 32, True, True, 65),
    ("nvfp4", "f32", 6, 2, 128, 64, True, True, 19),
    ("int4_per_token_head", "f32", 3, 1, 128, 128, False, False, 40),
    ("fp8_per_token_head", "f32", 2, 2, 128, 0, False, True, 9),
]


def make_qkv(T, Hq, Hkv, D, dt, seed=11):
    """q, k, v as slices of one projection's rows (with 16 bytes of something else behind them)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, (Hq + 2 * Hkv) * D + 16))
    x[::7] *= 9.0
    x[3::11] *= 1e-3
    if T > 4:
        x[4, :D] = 0.0  # a head of zeros: eps alone
    t = torch.from_numpy(x).to(dt).cuda()
    cut = [0, Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D]
    return [t[:, a:b].unflatten(1, (-1, D)) for a, b in zip(cut, cut[1:])]


@pytest.mark.gpu
@pytest.mark.parametrize("mode,io,Hq,Hkv,D,rot,interleaved,norm,T", CASES)
def test_norm_rope_write(mode, io, Hq, Hkv, D, rot, interleaved, norm, T):
    K = kvq()
    dt = torch.float16 if io == "f16" else torch.float32
    ndt = np.float16 if io == "f16" else np.float32
    rng = np.random.default_rng(T)
    q, k, v = make_qkv(T, Hq, Hkv, D, dt)
    wq, wk = (torch.from_numpy(1.0 + 0.3 * rng.standard_normal(D)).to(dt).cuda() if norm else None for _ in range(2))
    pos = rng.integers(0, 5000, T).astype(np.int32)
    ang = np.arange(5000)[:, None] * 10000.0 ** (-np.arange(max(rot // 2, 1)) / max(rot // 2, 1))
    tab = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    pages = (T + 15) // 16 + 2
    cfg = K.make_config(pages, 16, Hkv, D, mode, dt)
    pools = [guarded(K.kvq_cache_bytes(cfg), torch.uint8, fill=0xCD, name="pool") for _ in range(2)]
    caches = [K.kvq_cache_alloc(cfg, p) for p in pools]
    if mode in TENSOR_SCALED:
        for c in caches:
            K.kvq_cache_set_tensor_scales(c, 0.02, 0.015)
    slots = rng.permutation(pages * 16)[:T].astype(np.int32)
    slots[:T // 2] = np.sort(slots[:T // 2])  # runs and strays
    if T > 8:
        slots[5] = -1
    sd = torch.from_numpy(slots).cuda()
    q_out = guarded((T, Hq, D), dt, fill=5.0, name="q_out")
    k_out = guarded((T, Hkv, D), dt, fill=5.0, name="k_out")
    td = torch.from_numpy(tab).cuda() if rot else None
    K.kvq_norm_rope_write(caches[0], q, k, v, torch.from_numpy(pos).cuda(), td, q_out, slot_mapping=sd, k_out=k_out,
                          q_weight=wq, k_weight=wk, eps=1e-5, interleaved=interleaved)
    torch.cuda.synchronize()
    assert K.kvq_cache_read_errors(caches[0]) == 0
    for x, w, out in ((q, wq, q_out), (k, wk, k_out)):
        z = rotated(x.cpu().numpy(), None if w is None else w.cpu().numpy(), tab[pos], rot, interleaved, 1e-5)
        got, want = out.cpu().numpy(), z.astype(ndt)
        differ = got != want
        assert not (differ & ~near_border(z, ndt)).any(), f"{differ.sum()} values are not the rounded formula"
    # the pool: what a plain write of the rotated keys and the values stores, bit for bit
    K.kvq_quantize_write(caches[1], k_out, v.contiguous(), sd)
    torch.cuda.synchronize()
    assert torch.equal(pools[0], pools[1])
    # in place, without the cache
    qi, ki = q.contiguous(), k.contiguous()
    K.kvq_norm_rope_write(caches[0], qi, ki, None, torch.from_numpy(pos).cuda(), td, qi, k_out=ki, q_weight=wq,
                          k_weight=wk, eps=1e-5, interleaved=interleaved)
    assert torch.equal(qi, q_out) and torch.equal(ki, k_out)


@pytest.mark.gpu
def test_norm_rope_positions_and_refusals():
    K = kvq()
    cfg = K.make_config(4, 16, 2, 128, "int8_per_token_head", torch.float16)
    pool = guarded(K.kvq_cache_bytes(cfg), torch.uint8, fill=0xCD, name="pool")
    cache = K.kvq_cache_alloc(cfg, pool)
    q, k, v = make_qkv(6, 4, 2, 128, torch.float16)
    tab = torch.ones(8, 128, device="cuda")
    pos = torch.tensor([0, 8, 1, -1, 7, 2], dtype=torch.int32, device="cuda")
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    out = guarded((6, 4, 128), torch.float16, fill=3.0, name="q_out")
    K.kvq_norm_rope_write(cache, q, k, v, pos, tab, out, slot_mapping=slots)
    torch.cuda.synchronize()
    assert K.kvq_cache_read_errors(cache) == 0x80
    assert (out[[1, 3]] == 3.0).all() and not (out[[0, 2, 4, 5]] == 3.0).all(-1).any()
    rows = pool[256:].view(4, 2, -1)[0, :, :16 * 128].view(2, 16, 128)
    assert (rows[:, [1, 3]] == 0xCD).all() and not (rows[:, [0, 2, 4, 5]] == 0xCD).all(-1).any()

    ok = dict(slot_mapping=slots)
    bad = [
        (ValueError, (q.float(), k, v, pos, tab, out), ok),
        (ValueError, (q, k, v, pos.long(), tab, out), ok),
        (ValueError, (q, k[:, :1], v, pos, tab, out), ok),
        (ValueError, (q.transpose(1, 2).contiguous().transpose(1, 2), k, v, pos, tab, out), ok),
        (ValueError, (q, k, v, pos, tab, out), dict(slot_mapping=slots[:5])),
        (ValueError, (q, k, v, pos, tab, out), dict(slot_mapping=slots, q_weight=tab[0])),
        (K.KVQError, (q, k, v, pos, torch.ones(8, 24, device="cuda"), out), ok),   # rot_dim 24
        (K.KVQError, (q, k, v, pos, torch.ones(8, 144, device="cuda"), out), ok),  # rot_dim > head_dim
        (K.KVQError, (q, k, v, pos, tab, out), dict(slot_mapping=slots, eps=-1.0)),
        (K.KVQError, (q, k, None, pos, tab, out), ok),                             # a write without values
        (K.KVQError, (q, k, v, pos, tab, out), dict(slot_mapping=slots, mode="nvfp4")),
    ]
    for err, args, kw in bad:
        with pytest.raises(err):
            K.kvq_norm_rope_write(cache, *args, **kw)
    wide = torch.zeros(6, 4 * 128 + 4, dtype=torch.float16, device="cuda")  # rows 8 bytes off
    with pytest.raises(K.KVQError):
        K.kvq_norm_rope_write(cache, wide[:, :512].unflatten(1, (4, 128)), k, v, pos, tab, out, **ok)
    kcfg = K.make_config(1, 128, 2, 128, "kvarn_k4v2_g128", torch.float16)
    kc = K.kvq_cache_alloc(kcfg, torch.zeros(K.kvq_cache_bytes(kcfg), dtype=torch.uint8, device="cuda"))
    with pytest.raises(K.KVQError) as e:
        K.kvq_norm_rope_write(kc, q, k, v, pos, tab, out, **ok)
    assert e.value.status == 2
    torch.cuda.synchronize()
    assert K.kvq_cache_read_errors(cache) == 0  # nothing of the refused calls ran


@pytest.mark.gpu
def test_norm_rope_then_append_and_read_kvarn():
    """A KVarN cache takes the rotated keys by its own write; they read back within its quantization."""
    K = kvq()
    cfg = K.make_config(2, 128, 2, 128, "kvarn_k4v2_g128", torch.float16)
    pool = guarded(K.kvq_cache_bytes(cfg), torch.uint8, fill=0, name="pool")
    cache = K.kvq_cache_alloc(cfg, pool)
    q, k, v = make_qkv(256, 4, 2, 128, torch.float16)
    w = torch.ones(128, dtype=torch.float16, device="cuda")
    pos = torch.arange(256, dtype=torch.int32, device="cuda")
    tab = torch.cat([torch.cos(pos[:, None] * 0.01 * torch.arange(64, device="cuda")),
                     torch.sin(pos[:, None] * 0.01 * torch.arange(64, device="cuda"))], 1)
    q_out, k_out = torch.empty_like(q), torch.empty_like(k)
    K.kvq_norm_rope_write(cache, q, k, None, pos, tab, q_out.contiguous(), k_out=(ko := k_out.contiguous()), k_weight=w)
    vc = v.contiguous()
    K.kvq_quantize_write(cache, ko, vc, pos)
    back_k, back_v = (guarded((256, 2, 128), torch.float32, fill=0.0, name="out") for _ in range(2))
    K.kvq_cache_read(cache, pos, back_k, back_v)
    pool_h = pool.cpu().numpy()
    ref = pool_values("kvarn_k4v2_g128", pool_h, 2, 2, 128, 1.0, 1.0).reshape(2, 256, 2, 128)
    for got, want in ((back_k, ref[0]), (back_v, ref[1])):
        tol = 16 * 2.0 ** -24 * np.linalg.norm(want, axis=-1, keepdims=True) * 11.4 + 2.0 ** -25
        assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    st = oracle  # the oracle module stays importable beside the library
    assert st is not None


@pytest.mark.gpu
def test_captured_step_replays():
    """Write and read captured into one graph on a side stream, replayed on new inputs."""
    K = kvq()
    cfg = K.make_config(4, 16, 2, 128, "nvfp4", torch.float16)
    pool = guarded(K.kvq_cache_bytes(cfg), torch.uint8, fill=0, name="pool")
    cache = K.kvq_cache_alloc(cfg, pool)
    K.kvq_cache_set_tensor_scales(cache, 0.01, 0.01)
    q, k, v = (x.contiguous() for x in make_qkv(20, 4, 2, 128, torch.float16))
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    slots = pos + 7
    tab = torch.ones(32, 128, device="cuda") * 0.5
    q_out, kr, vr = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)

    def step():
        K.kvq_norm_rope_write(cache, q, k, v, pos, tab, q_out, slot_mapping=slots)
        K.kvq_cache_read(cache, slots, kr, vr)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    for x in (q, k, v):
        x.mul_(-2.0)
    g.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (q_out, kr, vr)]
    step()
    torch.cuda.synchronize()
    for a, b in zip(got, (q_out, kr, vr)):
        assert torch.equal(a, b)
    assert K.kvq_cache_read_errors(cache) == 0

"""What the serving operators around the paged cache are measured on: three
calls that take a prompt chunk (or one token per sequence) through the cache.

* read: ``kvq_cache_read`` -- the values the cache holds at given slots.
* write: ``kvq_norm_rope_write`` -- per-head RMS norm and position rotation of
  queries and keys, then the quantized write of keys and values, in one pass.
  The cache's new contents come back as the values they stand for, through
  ``kvq_cache_read``.
* attend: ``kvq_chunk_attention`` -- ragged chunks of new tokens (a chunk of
  one is a decode step) over the paged cache, with a capped score, a bias by
  distance, a sliding window or a bidirectional prefix.

With ``own`` false, ``run`` computes the same in elementary torch operations
from the same packed pages; sizes follow the repository's workloads (64/8 and
32/8 heads of 128, 4 heads of 32; contexts up to 32768; 16- and 128-token
pages; outlier tokens and channels).
"""
import math
import random

import torch

own = False

PAGE = {"kvarn_k4v2_g128": 128}
MODES = ["fp8_per_tensor", "int8_per_token_head", "fp8_per_token_head", "nvfp4", "int4_per_token_head"]


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a few scattered tokens looked at by a scheduler or a test of the cache: latency
        dict(name="read_200_int8", op="read", mode="int8_per_token_head", io="f16", tokens=200, kv_heads=8, dim=128),
        # a long context expanded for a consumer that wants dense keys and values
        dict(name="read_64k_nvfp4", op="read", mode="nvfp4", io="f16", tokens=65521, kv_heads=8, dim=128),
        # the same from rotated 128-token tiles
        dict(name="read_12k_kvarn", op="read", mode="kvarn_k4v2_g128", io="f16", tokens=12801, kv_heads=8, dim=128),
        # one decode step of 64 sequences: latency
        dict(name="write_step_64_fp8", op="write", mode="fp8_per_token_head", io="f16", tokens=64, heads=64, kv_heads=8,
             dim=128, rot=128, interleaved=False, norm=True),
        # a prompt chunk of 8K tokens
        dict(name="write_8k_int8", op="write", mode="int8_per_token_head", io="f16", tokens=8191, heads=64, kv_heads=8,
             dim=128, rot=128, interleaved=False, norm=True),
        # fp32 activations, half of each head rotated in neighbouring pairs, 4-bit cache
        dict(name="write_2k_nvfp4_f32", op="write", mode="nvfp4", io="f32", tokens=2047, heads=32, kv_heads=8, dim=128,
             rot=64, interleaved=True, norm=True),
        # prompts from their first token, three sequences of different lengths
        dict(name="attend_prompt_int8", op="attend", mode="int8_per_token_head", io="f16", seqs=3, q_lo=700, q_hi=2048,
             ctx_lo=0, ctx_hi=0, heads=32, kv_heads=8, dim=128, cap=0.0, alibi=False, window=0, prefix=False, shape=1),
        # a 2K chunk of a prompt whose first 30K tokens are in the cache
        dict(name="attend_2k_of_32k_nvfp4", op="attend", mode="nvfp4", io="f16", seqs=1, q_lo=2048, q_hi=2048,
             ctx_lo=30720, ctx_hi=30720, heads=64, kv_heads=8, dim=128, cap=0.0, alibi=False, window=0, prefix=False,
             shape=2),
        # short chunks (a few drafted tokens, the ends of prompts) of 16 sequences, scores capped, local layers
        dict(name="attend_short_fp8_window", op="attend", mode="fp8_per_tensor", io="f16", seqs=16, q_lo=1, q_hi=60,
             ctx_lo=500, ctx_hi=8000, heads=32, kv_heads=8, dim=128, cap=50.0, alibi=False, window=4096, prefix=False,
             shape=3),
        # single tokens of 32 sequences with capped scores
        dict(name="attend_step_32_fp8_cap", op="attend", mode="fp8_per_token_head", io="f16", seqs=32, q_lo=1, q_hi=1,
             ctx_lo=1000, ctx_hi=16000, heads=64, kv_heads=8, dim=128, cap=30.0, alibi=False, window=0, prefix=False,
             shape=4),
        # two single tokens with a bias by distance: latency
        dict(name="attend_step_2_int4_alibi", op="attend", mode="int4_per_token_head", io="f16", seqs=2, q_lo=1, q_hi=1,
             ctx_lo=100, ctx_hi=400, heads=32, kv_heads=8, dim=128, cap=0.0, alibi=True, window=0, prefix=False, shape=5),
        # fp32 heads of 32 with a bidirectional prefix
        dict(name="attend_prefix_int8_f32", op="attend", mode="int8_per_token_head", io="f32", seqs=4, q_lo=60, q_hi=300,
             ctx_lo=0, ctx_hi=900, heads=4, kv_heads=4, dim=32, cap=0.0, alibi=False, window=0, prefix=True, shape=6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["read", "write", "attend", "attend", "attend"])
    if op == "read":
        mode = rng.choice(MODES + ["kvarn_k4v2_g128"])
        return dict(op=op, mode=mode, io=rng.choice(["f16", "f16", "f32"]), tokens=_log_int(rng, 1, 32768),
                    kv_heads=rng.choice([1, 4, 8]), dim=128 if mode.startswith("kvarn") else rng.choice([32, 128, 128]))
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 3, 4, 7, 8])
    dim = rng.choice([32, 128, 128, 128])
    if op == "write":
        return dict(op=op, mode=rng.choice(MODES), io=rng.choice(["f16", "f16", "f32"]), tokens=_log_int(rng, 1, 8191),
                    heads=kv * group, kv_heads=kv, dim=dim, rot=rng.choice([dim, dim // 2]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8)
    kind = rng.choice(["step", "short", "long"])
    io = rng.choice(["f16", "f16", "f16", "f32"])
    c = dict(op=op, mode=rng.choice(MODES), io=io, heads=kv * group, kv_heads=kv, dim=dim)
    if kind == "step":
        c.update(seqs=_log_int(rng, 1, 32), q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=_log_int(rng, 20, 16000))
    elif kind == "short":
        c.update(seqs=_log_int(rng, 1, 16), q_lo=1, q_hi=_log_int(rng, 2, 100), ctx_lo=0, ctx_hi=_log_int(rng, 20, 8000))
    else:
        q = _log_int(rng, 100, 2048)
        c.update(seqs=rng.randint(1, 3), q_lo=max(1, q // 3), q_hi=q, ctx_lo=0, ctx_hi=_log_int(rng, 1, 6000))
    extra = rng.choice(["none", "cap", "alibi", "window", "prefix", "cap+window", "prefix+window"])
    c.update(cap=rng.choice([20.0, 50.0]) if "cap" in extra else 0.0, alibi=extra == "alibi",
             window=_log_int(rng, 1, 4096) if "window" in extra else 0, prefix="prefix" in extra,
             shape=rng.randrange(1 << 20))
    return c


def _lens(case):
    """Per sequence: (new tokens, all tokens, prefix) -- the shape is the case's, the values are the seed's."""
    r = random.Random(case["shape"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    n = [a + r.randint(case["ctx_lo"], case["ctx_hi"]) for a in q]
    p = [r.randint(0, b) if case["prefix"] else 0 for b in n]
    return q, n, p


def _row_bytes(mode, dim):
    """Bytes of one token of one kv head, keys and values, scales included."""
    return {"fp8_per_tensor": 2 * dim, "int8_per_token_head": 2 * dim + 8, "fp8_per_token_head": 2 * dim + 8,
            "nvfp4": dim + dim // 8, "int4_per_token_head": dim + 8, "kvarn_k4v2_g128": dim}[mode]


def work(case):
    e = 2 if case["io"] == "f16" else 4
    D, K = case["dim"], case["kv_heads"]
    packed = _row_bytes(case["mode"], D) * K
    if case["op"] == "read":
        return {"bytes": case["tokens"] * (packed + 2 * K * D * e + 4), "flops": case["tokens"] * K * D * 4}
    if case["op"] == "write":  # q in and out, k and v in, the packed rows out; then the packed rows in, the values out
        row = 2 * case["heads"] * D * e + 2 * K * D * e + packed + 8 + 4 * case["rot"]
        return {"bytes": case["tokens"] * (row + packed + 2 * K * D * e + 4),
                "flops": case["tokens"] * (case["heads"] + 2 * K) * D * 8}
    q, n, p = _lens(case)
    bytes_, pairs = 0, 0
    for a, b, f in zip(q, n, p):
        first = b - a  # position of the chunk's first token
        w = case["window"] or b
        lo = max(0, first - w + 1)
        kept = b - lo + min(f, lo)
        bytes_ += 2 * a * case["heads"] * D * e + kept * packed
        for t in range(first, b):
            s = max(0, t - w + 1)
            pairs += t + 1 - s + max(0, min(f, s)) + max(0, f - t - 1)
    return {"bytes": bytes_, "flops": 4 * pairs * case["heads"] * D}


# ---------------------------------------------------------------- packed pages, in torch
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _block_bytes(mode, P, D):
    return P * _row_bytes(mode, D) if mode != "kvarn_k4v2_g128" else P * D * 3 // 4 + 4 * (3 * D + P) + 4 * (3 * P + D)


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _e2m1_code(x):
    """Nearest E2M1 magnitude, ties to the even code, the sign in bit 3."""
    a = x.abs()
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5.0).int())
    return c + 8 * (torch.signbit(x) & (a >= 0)).int()


def _quantize(x, mode, scale):
    """x fp32 [.., D] -> (codes, scales): codes int32, or float8 for the E4M3 payloads."""
    if mode == "fp8_per_tensor":
        return _e4m3(x / scale), None
    if mode in ("int8_per_token_head", "int4_per_token_head", "fp8_per_token_head"):
        top = {"int8_per_token_head": 127.0, "int4_per_token_head": 7.0, "fp8_per_token_head": 448.0}[mode]
        s = x.abs().amax(-1, keepdim=True).clamp_min(1e-8) / torch.tensor(top, device=x.device)
        if mode == "fp8_per_token_head":
            return _e4m3(x / s), s
        return torch.round(x / s).clamp(-top, top).int(), s
    b = x.unflatten(-1, (-1, 16))
    st = torch.tensor(scale, dtype=torch.float32, device=x.device)
    sb = _e4m3(b.abs().amax(-1, keepdim=True) / (6.0 * st))
    den = st * sb.float()
    return torch.where(den > 0, _e2m1_code(b / torch.where(den > 0, den, 1.0)), 0).flatten(-2), sb.squeeze(-1)


def _value(codes, scales, mode, scale):
    """The values that codes and scales stand for, fp32."""
    if mode == "fp8_per_tensor":
        return codes.float() * scale
    if mode != "nvfp4":
        return codes.float() * scales
    lut = torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device)
    v = lut[codes.int()].unflatten(-1, (-1, 16))
    return (v * (scales.float() * scale).unsqueeze(-1)).flatten(-2)


def _bytes(x):
    return x.contiguous().view(torch.uint8)


def _pack(k, v, mode, ks, vs):
    """Pages [N, H, P, D] of fp32 keys and values -> [N, H, block bytes]."""
    N, H, P, D = k.shape
    (kc, ksc), (vc, vsc) = _quantize(k, mode, ks), _quantize(v, mode, vs)
    flat = lambda x: _bytes(x).reshape(N, H, -1)  # noqa: E731
    if mode == "fp8_per_tensor":
        return torch.cat([flat(kc), flat(vc)], -1)
    if mode in ("int8_per_token_head", "fp8_per_token_head"):
        if mode == "int8_per_token_head":
            kc, vc = kc.to(torch.int8), vc.to(torch.int8)
        return torch.cat([flat(kc), flat(vc), flat(ksc), flat(vsc)], -1)
    kc, vc = (kc & 15).to(torch.uint8), (vc & 15).to(torch.uint8)
    if mode == "nvfp4":
        kb = kc[..., 0::2] | (kc[..., 1::2] << 4)
        vb = vc[:, :, 0::2] | (vc[:, :, 1::2] << 4)
    else:
        n = kc.reshape(N, H, P, D // 8, 8)[..., [0, 2, 4, 6, 1, 3, 5, 7]]
        kb = n[..., 0::2] | (n[..., 1::2] << 4)
        n = vc.reshape(N, H, P // 2, 2, D // 4, 4).permute(0, 1, 2, 4, 3, 5).reshape(N, H, P // 2, D // 4, 8)
        vb = n[..., 0::2] | (n[..., 1::2] << 4)
    return torch.cat([flat(kb), flat(vb), flat(ksc), flat(vsc)], -1)


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2).int()


def _hadamard(n, device, dtype):
    i = torch.arange(n, device=device)
    b = i[:, None] & i[None, :]
    ones = sum((b >> s) & 1 for s in range(n.bit_length() - 1))
    return (1 - 2 * (ones % 2)).to(dtype) / math.sqrt(n)


def _unpack(blk, mode, P, D, ks, vs):
    """Blocks [..., block bytes] -> keys and values [..., P, D], fp32 (KVarN: still rotated)."""
    lead = blk.shape[:-1]
    part = lambda a, n: blk[..., a:a + n].contiguous()  # noqa: E731
    f32 = lambda a, n: part(a, 4 * n).view(torch.float32)  # noqa: E731
    if mode in ("fp8_per_tensor", "int8_per_token_head", "fp8_per_token_head"):
        t = torch.int8 if mode == "int8_per_token_head" else torch.float8_e4m3fn
        k, v = (part(s * P * D, P * D).view(t).reshape(*lead, P, D) for s in (0, 1))
        if mode == "fp8_per_tensor":
            return _value(k, None, mode, ks), _value(v, None, mode, vs)
        a, b = (f32(2 * P * D + 4 * P * s, P).unsqueeze(-1) for s in (0, 1))
        return _value(k, a, mode, ks), _value(v, b, mode, vs)
    if mode == "kvarn_k4v2_g128":
        k = _nibbles(part(0, P * D // 2)).reshape(*lead, P, D).float()
        v = part(P * D // 2, P * D // 4)
        v = torch.stack([(v >> s) & 3 for s in (0, 2, 4, 6)], -1).reshape(*lead, P, D).float()
        m = P * D * 3 // 4
        sc, z, c, r = f32(m, D), f32(m + 4 * D, D), f32(m + 8 * D, D), f32(m + 12 * D, P)
        k = r.unsqueeze(-1) * c.unsqueeze(-2) * (sc.unsqueeze(-2) * k + z.unsqueeze(-2))
        m += 4 * (3 * D + P)
        sc, z, r, c = f32(m, P), f32(m + 4 * P, P), f32(m + 8 * P, P), f32(m + 12 * P, D)
        return k, r.unsqueeze(-1) * c.unsqueeze(-2) * (sc.unsqueeze(-1) * v + z.unsqueeze(-1))
    kn, vn = _nibbles(part(0, P * D // 2)), _nibbles(part(P * D // 2, P * D // 2))
    if mode == "nvfp4":
        k = kn.reshape(*lead, P, D)
        v = vn.reshape(*lead, P // 2, D, 2).transpose(-1, -2).reshape(*lead, P, D)
        a, b = (part(P * D + s * P * D // 16, P * D // 16).view(torch.float8_e4m3fn).reshape(*lead, P, D // 16) for s in (0, 1))
    else:
        k = kn.reshape(*lead, P, D // 8, 8)[..., [0, 4, 1, 5, 2, 6, 3, 7]].reshape(*lead, P, D)
        v = vn.reshape(*lead, P // 2, D // 4, 2, 4).transpose(-3, -2).reshape(*lead, P, D)
        k, v = (k ^ 8) - 8, (v ^ 8) - 8
        a, b = (f32(P * D + 4 * P * s, P).unsqueeze(-1) for s in (0, 1))
    return _value(k, a, mode, ks), _value(v, b, mode, vs)


# ---------------------------------------------------------------- inputs
def _io(case):
    return torch.float16 if case["io"] == "f16" else torch.float32


def _pool(case, pages, gen):
    """A filled pool of `pages` pages: standard normal keys and values, some tokens and channels larger, as in the
    repository's workloads."""
    mode, H, D = case["mode"], case["kv_heads"], case["dim"]
    P = PAGE.get(mode, 16)
    ks = vs = 1.0
    body = torch.empty(pages, H, _block_bytes(mode, P, D), dtype=torch.uint8, device="cuda")
    if mode == "kvarn_k4v2_g128":
        codes = torch.randint(0, 256, (pages, H, P * D * 3 // 4), dtype=torch.uint8, device="cuda", generator=gen)
        def f(n, lo, hi): return torch.rand(pages, H, n, device="cuda", generator=gen) * (hi - lo) + lo  # noqa: E704
        meta = [f(D, 0.25, 0.45), f(D, -3.0, -2.0), f(D, 0.5, 2.0), f(P, 0.7, 1.4),
                f(P, 1.0, 1.6), f(P, -3.0, -2.0), f(P, 0.7, 1.4), f(D, 0.5, 2.0)]
        body.copy_(torch.cat([codes] + [_bytes(m).reshape(pages, H, -1) for m in meta], -1))
    else:
        if mode == "fp8_per_tensor":
            ks = vs = 20.0 * 4.5 / 448.0  # sink tokens x20
        elif mode == "nvfp4":
            ks = vs = 10.0 * 4.5 / 2688.0  # channels x10
        for a in range(0, pages, 1 << 12):
            n = min(1 << 12, pages - a)
            kv = []
            for _ in range(2):
                x = torch.randn(n, H, P, D, device="cuda", generator=gen)
                if mode == "fp8_per_tensor":
                    x = torch.where(torch.rand(n, H, P, 1, device="cuda", generator=gen) < 0.002, 20.0 * x, x)
                elif mode == "nvfp4":
                    x[..., 3::61] *= 10.0
                kv.append(x.to(_io(case)).float())
            body[a:a + n] = _pack(kv[0], kv[1], mode, ks, vs)
    pool = torch.zeros(256 + body.numel(), dtype=torch.uint8, device="cuda")
    pool[256:] = body.flatten()
    return pool, ks, vs


def _open(case, st, pages):
    """What a program keeps of the library: the cache handle over the pool."""
    from quantized_paged_kv_quantize_gb300 import kvq
    cfg = kvq.make_config(pages, st["P"], case["kv_heads"], case["dim"], case["mode"], _io(case))
    st["kvq"] = kvq
    st["cache"] = kvq.kvq_cache_alloc(cfg, st["pool"])
    if case["mode"] in ("fp8_per_tensor", "nvfp4"):
        kvq.kvq_cache_set_tensor_scales(st["cache"], st["ks"], st["vs"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, D, H = _io(case), case["dim"], case["kv_heads"]
    P = PAGE.get(case["mode"], 16)
    st = dict(case=case, P=P)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    if case["op"] in ("read", "write"):
        T = case["tokens"]
        pages = (T + P - 1) // P + 3
        # whole sequences on scattered pages: tokens run through each page in order
        perm = torch.randperm(pages, device="cuda", generator=gen)
        t = torch.arange(T, device="cuda")
        st["slots"] = (perm[t // P] * P + t % P).int()
        if case["op"] == "read":
            st["pool"], st["ks"], st["vs"] = _pool(case, pages, gen)
        else:
            st["pool"] = torch.zeros(256 + pages * H * _block_bytes(case["mode"], P, D), dtype=torch.uint8, device="cuda")
            amax = 12.0
            st["ks"] = st["vs"] = amax / (448.0 if case["mode"] == "fp8_per_tensor" else 2688.0)
            hq = case["heads"]
            # one projection's rows: queries, keys, values of a token side by side
            qkv = randn(T, (hq + 2 * H) * D)
            qkv[::97] *= 4.0
            st["qkv"] = qkv.to(dt)
            st["wq"], st["wk"] = ((1.0 + 0.2 * randn(D)).to(dt) if case["norm"] else None for _ in range(2))
            span = 32768
            st["positions"] = torch.randint(0, span, (T,), device="cuda", generator=gen).int()
            half = case["rot"] // 2
            inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
            ang = torch.arange(span, device="cuda", dtype=torch.float64)[:, None] * inv
            st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], -1).float()
            st["q_out"] = torch.empty(T, hq, D, dtype=dt, device="cuda")
        st["k_out"], st["v_out"] = (torch.empty(T, H, D, dtype=dt, device="cuda") for _ in range(2))
    else:
        q, n, p = _lens(case)
        per = [(x + P - 1) // P for x in n]
        pages = sum(per) + 2
        st["pool"], st["ks"], st["vs"] = _pool(case, pages, gen)
        perm = torch.randperm(pages, device="cuda", generator=gen).int()
        st["table"] = torch.zeros(len(q), max(per), dtype=torch.int32, device="cuda")
        at = 0
        for b, m in enumerate(per):
            st["table"][b, :m] = perm[at:at + m]
            at += m
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        st["seq_lens"], st["prefix"] = ints(n), ints(p) if case["prefix"] else None
        st["cu"] = ints([sum(q[:b]) for b in range(len(q) + 1)])
        st["max_q"], st["max_n"] = max(q), max(n)
        st["q"] = randn(sum(q), case["heads"], D).to(dt)
        st["out"] = torch.empty_like(st["q"])
        st["slopes"] = None
        if case["alibi"]:
            st["slopes"] = 2.0 ** (-8.0 * torch.arange(1, case["heads"] + 1, device="cuda") / case["heads"])
    if own:
        _open(case, st, pages)
        if case["op"] == "attend":
            _, _, ws = st["kvq"].kvq_chunk_plan(st["cache"], st["q"].shape[0], len(q), case["heads"], max_q_len=st["max_q"],
                                                max_seq_len=st["max_n"], window=case["window"], has_prefix=case["prefix"])
            st["ws"] = torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if case["op"] == "read":
        if own:
            st["kvq"].kvq_cache_read(st["cache"], st["slots"], st["k_out"], st["v_out"])
            return st["k_out"], st["v_out"]
        return _plain_read(st, st["slots"])
    if case["op"] == "write":
        T, D, H, hq = case["tokens"], case["dim"], case["kv_heads"], case["heads"]
        q, k, v = (x.unflatten(1, (-1, D)) for x in st["qkv"].split([hq * D, H * D, H * D], 1))
        if own:
            K = st["kvq"]
            K.kvq_norm_rope_write(st["cache"], q, k, v, st["positions"], st["cos_sin"], st["q_out"],
                                  slot_mapping=st["slots"], q_weight=st["wq"], k_weight=st["wk"], eps=1e-6,
                                  interleaved=case["interleaved"])
            K.kvq_cache_read(st["cache"], st["slots"], st["k_out"], st["v_out"])
            return st["q_out"], st["k_out"], st["v_out"]
        return _plain_write(st, q, k, v)
    if own:
        st["kvq"].kvq_chunk_attention(st["cache"], st["q"], st["cu"], st["table"], st["seq_lens"], st["out"],
                                      max_q_len=st["max_q"], max_seq_len=st["max_n"], logit_cap=case["cap"],
                                      alibi_slopes=st["slopes"], window=case["window"], prefix_lens=st["prefix"],
                                      workspace=st["ws"])
        return st["out"]
    return _plain_attend(st)


def _plain_read(st, slots):
    case, P = st["case"], st["P"]
    D, dt = case["dim"], _io(case)
    blk = st["pool"][256:].reshape(-1, case["kv_heads"], _block_bytes(case["mode"], P, D))
    s = slots.long()
    if case["mode"] == "kvarn_k4v2_g128":
        k, v = (x.transpose(1, 2).flatten(0, 1)[s] for x in _unpack(blk, case["mode"], P, D, 1.0, 1.0))
        h = _hadamard(D, k.device, torch.float32)
        return (k @ h).to(dt), (v @ h).to(dt)
    k, v = _unpack(blk, case["mode"], P, D, st["ks"], st["vs"])
    return tuple(x.transpose(1, 2).flatten(0, 1)[s].to(dt) for x in (k, v))


def _rotated(x, w, cs, rot, interleaved, dt):
    """RMS norm and rotation of [T, heads, D], in 64 bits because a last bit moves a code across its border; rounded
    once to the activations' type."""
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
    cos, sin = cs.double().unsqueeze(1).chunk(2, -1)
    y, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y.chunk(2, -1)
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1).to(dt)


def _plain_write(st, q, k, v):
    case, dt = st["case"], _io(st["case"])
    cs = st["cos_sin"][st["positions"].long()]
    q_out = _rotated(q, st["wq"], cs, case["rot"], case["interleaved"], dt)
    k_new = _rotated(k, st["wk"], cs, case["rot"], case["interleaved"], dt)
    back = [_value(*_quantize(x.float(), case["mode"], s), case["mode"], s).to(dt)
            for x, s in ((k_new, st["ks"]), (v, st["vs"]))]
    return q_out, back[0], back[1]


def _visible(st, maxq, S, B):
    """[B, 1, 1, maxq, S]: token s is seen by the sequence's query i."""
    case = st["case"]
    n = st["seq_lens"].long()[:, None, None]
    m = (st["cu"][1:] - st["cu"][:-1]).long()[:, None, None]
    pos = n - m + torch.arange(maxq, device="cuda")[:, None]
    s = torch.arange(S, device="cuda")
    see = s <= pos
    if case["window"]:
        see = see & (s > pos - case["window"])
    if st["prefix"] is not None:
        see = see | (s < st["prefix"].long()[:, None, None])
    return (see & (s < n) & (pos >= 0))[:, None, None], (pos - s)[:, None, None]


def _plain_attend(st):
    case, P = st["case"], st["P"]
    D, H, B = case["dim"], case["kv_heads"], case["seqs"]
    G, maxq = case["heads"] // H, st["max_q"]
    blk = st["pool"][256:].reshape(-1, H, _block_bytes(case["mode"], P, D))[st["table"].long()]
    k, v = _unpack(blk, case["mode"], P, D, st["ks"], st["vs"])  # [B, pages, H, P, D]
    k, v = (x.transpose(1, 2).reshape(B, H, -1, D) for x in (k, v))
    cu = st["cu"].long()
    row = cu[:-1, None] + torch.arange(maxq, device="cuda")  # [B, maxq]
    real = row < cu[1:, None]
    q = st["q"][row.clamp(max=st["q"].shape[0] - 1)].float().reshape(B, maxq, H, G, D).permute(0, 2, 3, 1, 4)
    s = (q.reshape(B, H, G * maxq, D) @ k.transpose(-1, -2)).reshape(B, H, G, maxq, -1) * D ** -0.5
    if case["cap"]:
        s = case["cap"] * torch.tanh(s / case["cap"])
    see, dist = _visible(st, maxq, k.shape[2], B)
    if case["alibi"]:
        s = s - st["slopes"].reshape(1, H, G, 1, 1) * dist.abs()
    s = s.masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    s = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    o = (s.reshape(B, H, G * maxq, -1) @ v).reshape(B, H, G, maxq, D) / s.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(B, maxq, H * G, D)[real].to(_io(case))


# ---------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"read": _exact_read, "write": _exact_write, "attend": _exact_attend}[case["op"]](case, st)


def _fp8(b):
    """E4M3 bytes -> fp64, from the format's definition."""
    b = b.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * 2.0 ** (e - 10).double())
    return torch.where(b >> 7 == 1, -mag, mag)


def _exact_rows(case, st, pages, side):
    """[pages, H, P, D] fp64 values of one side, written from the layout byte by byte (rotated back for KVarN)."""
    mode, P, D, H = case["mode"], st["P"], case["dim"], case["kv_heads"]
    blk = st["pool"][256:].reshape(-1, H, _block_bytes(mode, P, D))[pages]
    dev = blk.device
    t, d = torch.arange(P, device=dev)[:, None], torch.arange(D, device=dev)[None, :]
    byte = lambda i: blk[..., i.expand(P, D)].to(torch.int64)  # noqa: E731
    def f32(i):
        w = sum(byte(i + j) << (8 * j) for j in range(4)).to(torch.int32)
        return w.view(torch.float32).double()
    st_ = float(torch.tensor((st["ks"], st["vs"])[side], dtype=torch.float32))
    if mode == "fp8_per_tensor":
        return _fp8(byte(side * P * D + t * D + d)) * st_
    if mode in ("int8_per_token_head", "fp8_per_token_head"):
        c = byte(side * P * D + t * D + d)
        c = _fp8(c) if mode[0] == "f" else (c - 256 * (c >> 7)).double()
        return c * f32(2 * P * D + side * 4 * P + 4 * t + 0 * d)
    if mode == "nvfp4":
        c = byte(t * (D // 2) + d // 2) >> (4 * (d % 2)) if side == 0 else byte(P * D // 2 + (t // 2) * D + d) >> (4 * (t % 2))
        mag = torch.tensor(E2M1, dtype=torch.float64, device=dev)[c & 7]
        val = torch.where((c >> 3) & 1 == 1, -mag, mag)
        return val * _fp8(byte(P * D + side * (P * D // 16) + t * (D // 16) + d // 16)) * st_
    if mode == "int4_per_token_head":
        if side == 0:
            nib, base = (d % 8) // 2 + 4 * (d % 2) + 0 * t, t * (D // 2) + 4 * (d // 8)
        else:
            nib, base = d % 4 + 4 * (t % 2), P * D // 2 + (t // 2) * D + 4 * (d // 4)
        c = (byte(base + nib // 2) >> (4 * (nib % 2))) & 15
        return (c - 16 * (c >> 3)).double() * f32(P * D + side * 4 * P + 4 * t + 0 * d)
    m = P * D * 3 // 4
    if side == 0:
        c = ((byte(t * (D // 2) + d // 2) >> (4 * (d % 2))) & 15).double()
        y = f32(m + 4 * (3 * D + t) + 0 * d) * f32(m + 4 * (2 * D + d) + 0 * t) * (f32(m + 4 * d + 0 * t) * c + f32(m + 4 * (D + d) + 0 * t))
    else:
        m += 4 * (3 * D + P)
        c = ((byte(P * D // 2 + t * (D // 4) + d // 4) >> (2 * (d % 4))) & 3).double()
        y = f32(m + 4 * (2 * P + t) + 0 * d) * f32(m + 4 * (3 * P + d) + 0 * t) * (f32(m + 4 * t + 0 * d) * c + f32(m + 4 * (P + t) + 0 * d))
    return y @ _hadamard(D, dev, torch.float64)


def _exact_read(case, st):
    P, D, H = st["P"], case["dim"], case["kv_heads"]
    out = []
    for side in (0, 1):
        x = torch.empty(case["tokens"], H, D, dtype=torch.float64, device="cuda")
        for a in range(0, case["tokens"], 8192):
            s = st["slots"][a:a + 8192].long()
            pages, at = torch.unique(s // P, return_inverse=True)
            rows = _exact_rows(case, st, pages, side)
            x[a:a + 8192] = rows[at, :, s % P]
        out.append(x)
    return tuple(out)


def _exact_write(case, st):
    D, H, hq, rot = case["dim"], case["kv_heads"], case["heads"], case["rot"]
    x = st["qkv"].double()
    half = rot // 2
    out = []
    for at, heads, w in ((0, hq, st["wq"]), (hq * D, H, st["wk"])):
        y = x[:, at:at + heads * D].reshape(-1, heads, D).clone()
        if w is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / D + 1e-6) * w.double()
        z = y.clone()
        ang = st["cos_sin"][st["positions"].long()].double()
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
            c, s = ang[:, j, None], ang[:, half + j, None]
            z[..., a] = y[..., a] * c - y[..., b] * s
            z[..., b] = y[..., a] * s + y[..., b] * c
        out.append(z)
    # codes are whole numbers of a coarse grid: what they stand for has no 64-bit value of its own
    return out[0], None, None


def _exact_attend(case, st):
    q, n, p = _lens(case)
    D, H, P = case["dim"], case["kv_heads"], st["P"]
    G = case["heads"] // H
    if work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(sum(q), case["heads"], D, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(len(q)):
        pages = st["table"][b, :(n[b] + P - 1) // P].long()
        k, v = (_exact_rows(case, st, pages, side).transpose(1, 2).reshape(-1, H, D)[:n[b]] for side in (0, 1))
        tok = torch.arange(n[b], device="cuda")
        for h in range(H):
            for a in range(0, q[b], 512):
                m = min(512, q[b] - a)
                pos = n[b] - q[b] + a + torch.arange(m, device="cuda")[:, None, None]
                x = st["q"][at + a:at + a + m, h * G:(h + 1) * G].double()
                s = torch.einsum("igd,td->igt", x, k[:, h]) / math.sqrt(D)
                if case["cap"]:
                    s = case["cap"] * torch.tanh(s / case["cap"])
                if case["alibi"]:
                    s = s - st["slopes"][h * G:(h + 1) * G].double()[:, None] * (pos - tok).abs()
                seen = tok <= pos
                if case["window"]:
                    seen = seen & (pos - tok < case["window"])
                seen = (seen | (tok < p[b])).expand_as(s)
                s = torch.softmax(torch.where(seen, s, -math.inf), -1)
                out[at + a:at + a + m, h * G:(h + 1) * G] = torch.einsum("igt,td->igd", s, v[:, h])
        at += q[b]
    return out

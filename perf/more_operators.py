"""What the calls on a latent cache are measured on: one quantized latent vector
and one rotated key part a token, shared by all heads, in 16-token pages.

* write: ``kvq_latent_write`` -- RMS norm of the latent rows, rotation of the
  keys' and the queries' rotary parts, and the quantized write, in one pass.
  The cache's new contents come back as the values they stand for, through
  ``kvq_latent_read``.
* read: ``kvq_latent_read`` -- the rows the cache holds at given slots.
* attend: ``kvq_latent_attention`` -- the absorbed form: ragged chunks of
  queries in the latent space (a chunk of one is a decode step) over the paged
  latents, which are keys and values at once.
* prompt: ``kvq_latent_prompt_attention`` -- the expanded form: ragged prompts
  over keys and values of their own heads, with the shared rotary key part.

With ``own`` false, ``run`` computes the same in elementary torch operations
from the same bytes.
"""
import math
import random

import torch

own = False

P = 16          # tokens of a page
ROPE = 64       # rotary channels
NOPE = 128      # an expanded head's other key channels, and its values
MODES = ["fp8_per_tensor", "int8_per_token_head", "fp8_per_token_head", "nvfp4"]


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a few hundred scattered tokens expanded for a short prefix: latency
        dict(name="read_300_fp8", op="read", mode="fp8_per_token_head", io="f16", latent=512, tokens=300),
        # a long context's latents as dense rows, for the expanded form
        dict(name="read_64k_nvfp4", op="read", mode="nvfp4", io="f16", latent=512, tokens=65521),
        # one decode step of 40 sequences: latency
        dict(name="write_step_40_int8", op="write", mode="int8_per_token_head", io="f16", latent=512, tokens=40, heads=64,
             interleaved=False, norm=True),
        # a prompt chunk of 8K tokens
        dict(name="write_8k_fp8", op="write", mode="fp8_per_token_head", io="f16", latent=512, tokens=8191, heads=64,
             interleaved=True, norm=True),
        # fp32 activations, 4-bit latents of half the width
        dict(name="write_2k_nvfp4_f32", op="write", mode="nvfp4", io="f32", latent=256, tokens=2047, heads=20,
             interleaved=False, norm=True),
        # two single tokens over short contexts: latency
        dict(name="step_2_int8", op="attend", mode="int8_per_token_head", io="f16", latent=512, seqs=2, q_lo=1, q_hi=1,
             ctx_lo=100, ctx_hi=400, heads=20, causal=True, lse=False, shape=1),
        # a decode step with many heads a token
        dict(name="step_32_fp8", op="attend", mode="fp8_per_token_head", io="f16", latent=512, seqs=32, q_lo=1, q_hi=1,
             ctx_lo=1000, ctx_hi=16000, heads=128, causal=True, lse=False, shape=2),
        # a decode step of a large batch over a 4-bit cache, few heads
        dict(name="step_64_nvfp4", op="attend", mode="nvfp4", io="f16", latent=512, seqs=64, q_lo=1, q_hi=1, ctx_lo=1000,
             ctx_hi=16000, heads=20, causal=True, lse=False, shape=3),
        # a few drafted tokens of each sequence, log-sum-exps wanted
        dict(name="drafts_16_fp8", op="attend", mode="fp8_per_tensor", io="f16", latent=512, seqs=16, q_lo=1, q_hi=6,
             ctx_lo=500, ctx_hi=8000, heads=40, causal=True, lse=True, shape=4),
        # a 1K chunk of a prompt whose first 7K tokens are in the cache
        dict(name="chunk_1k_of_8k_int8", op="attend", mode="int8_per_token_head", io="f16", latent=512, seqs=1, q_lo=1024,
             q_hi=1024, ctx_lo=7168, ctx_hi=7168, heads=128, causal=True, lse=False, shape=5),
        # three short prompts from their first token
        dict(name="prompts_3", op="prompt", io="f16", seqs=3, q_lo=300, q_hi=1500, ctx_lo=0, ctx_hi=0, heads=32, causal=True,
             lse=False, shape=6),
        # a 2K chunk over 8K expanded keys
        dict(name="prompt_2k_of_8k", op="prompt", io="f16", seqs=1, q_lo=2048, q_hi=2048, ctx_lo=6144, ctx_hi=6144, heads=128,
             causal=True, lse=True, shape=7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["read", "write", "attend", "attend", "attend", "prompt", "prompt"])
    io = rng.choice(["f16", "f16", "f16", "f32"])
    latent = rng.choice([512, 512, 256])
    mode = rng.choice(MODES)
    if op == "read":
        return dict(op=op, mode=mode, io=io, latent=latent, tokens=_log_int(rng, 1, 65521))
    if op == "write":
        return dict(op=op, mode=mode, io=io, latent=latent, tokens=_log_int(rng, 1, 8191), heads=rng.choice([1, 8, 20, 64]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.8)
    heads = rng.choice([1, 5, 8, 20, 32, 40, 64, 128])
    c = dict(op=op, io=io, heads=heads, causal=rng.random() < 0.85, lse=rng.random() < 0.4, shape=rng.randrange(1 << 20))
    most = 1 if io == "f16" else 8  # (the fp32 form is for small work)
    if op == "prompt":
        q = _log_int(rng, 1, 2048 // most)
        c.update(seqs=rng.randint(1, 4), q_lo=max(1, q // 4), q_hi=q, ctx_lo=0, ctx_hi=_log_int(rng, 1, 4096 // most))
        return c
    c.update(mode=mode, latent=latent)
    kind = rng.choice(["step", "step", "drafts", "chunk"])
    if kind == "step":
        c.update(seqs=_log_int(rng, 1, 64 // most), q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=_log_int(rng, 20, 16000 // most))
    elif kind == "drafts":
        c.update(seqs=_log_int(rng, 1, 16), q_lo=0, q_hi=_log_int(rng, 2, 12), ctx_lo=0, ctx_hi=_log_int(rng, 20, 8000 // most))
    else:
        q = _log_int(rng, 13, 1024 // most)
        c.update(seqs=rng.randint(1, 3), q_lo=max(1, q // 3), q_hi=q, ctx_lo=0, ctx_hi=_log_int(rng, 1, 4000 // most))
    return c


def _lens(case):
    """Per sequence: (queries, all tokens) -- the shape is the case's, the values are the seed's."""
    r = random.Random(case["shape"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    if sum(q) == 0:
        q[0] = 1
    return q, [a + r.randint(case["ctx_lo"], case["ctx_hi"]) for a in q]


def _row_bytes(mode, latent):
    """Bytes of one token: codes, scales and the fp16 rotary part."""
    return 2 * ROPE + {"fp8_per_tensor": latent, "int8_per_token_head": latent + 4, "fp8_per_token_head": latent + 4,
                       "nvfp4": latent // 2 + latent // 16}[mode]


def work(case):
    e = 2 if case["io"] == "f16" else 4
    if case["op"] in ("read", "write"):
        L, T = case["latent"], case["tokens"]
        packed, row = _row_bytes(case["mode"], L), (L + ROPE) * e
        if case["op"] == "read":
            return {"bytes": T * (packed + row + 4), "flops": 2 * T * L}
        # rows, weights and angles in; queries, normed rows and packed rows out; then the packed rows in, the values out
        parts = 2 * case["heads"] * ROPE * e + 2 * row + packed + 8 + 4 * ROPE
        return {"bytes": T * (parts + packed + row + 4), "flops": T * (case["heads"] * ROPE * 3 + 8 * L)}
    q, n = _lens(case)
    pairs = sum(a * (b - a) + a * (a + 1) // 2 if case["causal"] else a * b for a, b in zip(q, n))
    H = case["heads"]
    if case["op"] == "attend":
        L = case["latent"]
        kept = sum(b for a, b in zip(q, n) if a)
        return {"bytes": sum(q) * H * (2 * L + ROPE) * e + kept * _row_bytes(case["mode"], L),
                "flops": 2 * pairs * H * (2 * L + ROPE)}
    return {"bytes": sum(q) * H * (2 * NOPE + ROPE) * e + sum(n) * (2 * H * NOPE + ROPE) * e,
            "flops": 2 * pairs * H * (2 * NOPE + ROPE)}


# ---------------------------------------------------------------- packed pages, in torch
# A page: codes [16][L] (NVFP4: [16][L / 2], the even channel in the low nibble), the rotary
# part [16][64] fp16, then the scales: [16] fp32, or NVFP4 [16][L / 16] E4M3.
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _e2m1_code(x):
    """Nearest E2M1 magnitude, ties to the even code, the sign in bit 3."""
    a = x.abs()
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5.0).int())
    return c + 8 * (torch.signbit(x) & (a >= 0)).int()


def _quantize(x, mode, scale):
    """x fp32 [.., L] -> (codes, scales)."""
    if mode == "fp8_per_tensor":
        return _e4m3(x / scale), None
    if mode != "nvfp4":
        top = 127.0 if mode == "int8_per_token_head" else 448.0
        s = x.abs().amax(-1, keepdim=True).clamp_min(1e-8) / torch.tensor(top, device=x.device)
        return (_e4m3(x / s) if top == 448.0 else torch.round(x / s).clamp(-top, top).to(torch.int8)), s
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
    v = lut[codes.long()].unflatten(-1, (-1, 16))
    return (v * (scales.float() * scale).unsqueeze(-1)).flatten(-2)


def _bytes(x):
    return x.contiguous().view(torch.uint8).reshape(x.shape[0], -1)


def _pack(c, kr, mode, scale):
    """Pages [N, P, L] and [N, P, ROPE] of fp32 rows -> [N, page bytes]."""
    codes, s = _quantize(c, mode, scale)
    if mode == "nvfp4":
        codes = (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)
    return torch.cat([_bytes(codes), _bytes(kr.half())] + ([] if s is None else [_bytes(s)]), -1)


def _unpack(blk, mode, L, scale):
    """Pages [.., page bytes] -> latents [.., P, L] and rotary parts [.., P, ROPE], fp32."""
    lead = blk.shape[:-1]
    n = P * L // 2 if mode == "nvfp4" else P * L
    part = lambda a, n: blk[..., a:a + n].contiguous()  # noqa: E731
    rope = part(n, 2 * P * ROPE).view(torch.float16).reshape(*lead, P, ROPE).float()
    at = n + 2 * P * ROPE
    if mode == "nvfp4":
        b = part(0, n)
        codes = torch.stack([b & 15, b >> 4], -1).reshape(*lead, P, L)
        s = part(at, P * L // 16).view(torch.float8_e4m3fn).reshape(*lead, P, L // 16)
    else:
        codes = part(0, n).view(torch.int8 if mode == "int8_per_token_head" else torch.float8_e4m3fn).reshape(*lead, P, L)
        s = None if mode == "fp8_per_tensor" else part(at, 4 * P).view(torch.float32).reshape(*lead, P, 1)
    return _value(codes, s, mode, scale), rope


# ---------------------------------------------------------------- inputs
def _io(case):
    return torch.float16 if case["io"] == "f16" else torch.float32


def _scale(mode):
    """A per-tensor scale: latents are normed, so their largest value is about 9."""
    return {"fp8_per_tensor": 9.0 / 448.0, "nvfp4": 9.0 / 2688.0}.get(mode, 1.0)


def _pool(case, pages, gen):
    """A filled pool: normed latents with a few larger channels, a few larger tokens."""
    mode, L = case["mode"], case["latent"]
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    pool = torch.zeros(256 + pages * P * _row_bytes(mode, L), dtype=torch.uint8, device="cuda")
    body = pool[256:].reshape(pages, -1)
    gain = torch.exp(0.3 * randn(L))
    for a in range(0, pages, 1 << 12):
        n = min(1 << 12, pages - a)
        c, kr = randn(n, P, L) * gain, 1.5 * randn(n, P, ROPE)
        c = torch.where(torch.rand(n, P, 1, device="cuda", generator=gen) < 0.004, 3.0 * c, c)
        body[a:a + n] = _pack(c, kr, mode, _scale(mode))
    return pool


def _open(case, st, pages):
    """What a program keeps of the library: the cache handle over the pool."""
    from quantized_paged_kv_quantize_gb300 import kvq
    st["kvq"] = kvq
    st["cache"] = kvq.kvq_latent_alloc(
        kvq.make_latent_config(pages, P, case.get("latent", 512), ROPE, case.get("mode", "fp8_per_token_head"), _io(case)),
        st["pool"])
    if case.get("mode") in ("fp8_per_tensor", "nvfp4"):
        kvq.kvq_latent_set_scale(st["cache"], _scale(case["mode"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _io(case)
    st = dict(case=case)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    empty = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    if case["op"] in ("read", "write"):
        T, L = case["tokens"], case["latent"]
        pages = (T + P - 1) // P + 3
        # whole sequences on scattered pages: tokens run through each page in order
        perm = torch.randperm(pages, device="cuda", generator=gen)
        t = torch.arange(T, device="cuda")
        st["slots"] = (perm[t // P] * P + t % P).int()
        if case["op"] == "read":
            st["pool"] = _pool(case, pages, gen)
        else:
            H = case["heads"]
            st["pool"] = torch.zeros(256 + pages * P * _row_bytes(case["mode"], L), dtype=torch.uint8, device="cuda")
            # one projection's rows: latent and rotary key part of a token side by side
            ckr = randn(T, L + ROPE)
            ckr[::97] *= 4.0
            st["ckr"] = ckr.to(dt)
            st["q"] = randn(T, H, NOPE + ROPE).to(dt)  # a head's rotary channels are its last
            st["w"] = (1.0 + 0.2 * randn(L)).to(dt) if case["norm"] else None
            st["positions"] = torch.randint(0, 32768, (T,), device="cuda", generator=gen).int()
            inv = 10000.0 ** (-torch.arange(ROPE // 2, device="cuda", dtype=torch.float64) / (ROPE // 2))
            ang = torch.arange(32768, device="cuda", dtype=torch.float64)[:, None] * inv
            st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], -1).float()
            st["q_out"] = torch.zeros(T, H, L + ROPE, dtype=dt, device="cuda")  # the absorbed queries' rows
            st["new"] = empty(T, L), empty(T, ROPE)
        st["back"] = empty(T, L), empty(T, ROPE)
        if own:
            _open(case, st, pages)
        return st
    q, n = _lens(case)
    H, T, S = case["heads"], sum(q), sum(n)
    st["cu"], st["seq_lens"] = ints([sum(q[:b]) for b in range(len(q) + 1)]), ints(n)
    st["max_q"], st["max_n"] = max(max(q), 1), max(n)
    st["scale"] = (NOPE + ROPE) ** -0.5
    st["lse"] = empty(T, H, dtype=torch.float32) if case["lse"] else None
    if case["op"] == "attend":
        L = case["latent"]
        per = [(x + P - 1) // P for x in n]
        pages = sum(per) + 2
        st["pool"] = _pool(case, pages, gen)
        perm = torch.randperm(pages, device="cuda", generator=gen).int()
        table, at = torch.zeros(len(q), max(per), dtype=torch.int32), 0
        perm = perm.cpu()
        for b, m in enumerate(per):
            table[b, :m] = perm[at:at + m]
            at += m
        st["table"] = table.cuda()
        st["q"] = (0.6 * randn(T, H, L + ROPE)).to(dt)
        st["out"] = empty(T, H, L)
        if own:
            _open(case, st, pages)
            _, ws = st["kvq"].kvq_latent_plan(st["cache"], T, len(q), H, max_q_len=st["max_q"], max_seq_len=st["max_n"])
            st["ws"] = empty(max(ws, 16), dtype=torch.uint8)
        return st
    st["cu_k"] = ints([sum(n[:b]) for b in range(len(q) + 1)])
    st["q"] = randn(T, H, NOPE + ROPE).to(dt)
    st["kv"] = randn(S, H, 2 * NOPE).to(dt)  # one projection's rows: a head's keys, then its values
    st["kr"] = (1.5 * randn(S, ROPE)).to(dt)
    st["out"] = empty(T, H, NOPE)
    if own:
        st["pool"] = torch.zeros(256 + P * _row_bytes("fp8_per_token_head", 512), dtype=torch.uint8, device="cuda")
        _open(case, st, 1)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if case["op"] == "read":
        if own:
            st["kvq"].kvq_latent_read(st["cache"], st["slots"], *st["back"])
            return st["back"]
        c, kr = _unpack(st["pool"][256:].reshape(-1, P * _row_bytes(case["mode"], case["latent"])), case["mode"],
                        case["latent"], _scale(case["mode"]))
        s = st["slots"].long()
        return c.flatten(0, 1)[s].to(_io(case)), kr.flatten(0, 1)[s].to(_io(case))
    if case["op"] == "write":
        if own:
            L, K = case["latent"], st["kvq"]
            K.kvq_latent_write(st["cache"], st["ckr"][:, :L], st["ckr"][:, L:], st["positions"], st["cos_sin"],
                               slot_mapping=st["slots"], q_rope=st["q"][..., NOPE:], q_rope_out=st["q_out"][..., L:],
                               latent_weight=st["w"], latent_out=st["new"][0], k_rope_out=st["new"][1], eps=1e-6,
                               interleaved=case["interleaved"])
            K.kvq_latent_read(st["cache"], st["slots"], *st["back"])
            return (st["q_out"][..., L:], *st["new"], *st["back"])
        return _plain_write(st)
    if own:
        if case["op"] == "attend":
            st["kvq"].kvq_latent_attention(st["cache"], st["q"], st["cu"], st["table"], st["seq_lens"], st["out"],
                                           max_q_len=st["max_q"], max_seq_len=st["max_n"], softmax_scale=st["scale"],
                                           causal=case["causal"], lse=st["lse"], workspace=st["ws"])
        else:
            st["kvq"].kvq_latent_prompt_attention(st["cache"], st["q"], st["kv"][..., :NOPE], st["kr"], st["kv"][..., NOPE:],
                                                  st["cu"], st["cu_k"], st["out"], max_q_len=st["max_q"],
                                                  max_k_len=st["max_n"], softmax_scale=st["scale"], causal=case["causal"],
                                                  lse=st["lse"])
        return (st["out"], st["lse"]) if case["lse"] else st["out"]
    return _plain_attend(st) if case["op"] == "attend" else _plain_prompt(st)


def _rotated(y, cs, interleaved, dt):
    """Rotation of the last ROPE channels of [T, heads, ROPE], in 64 bits because a last bit moves a code across its border."""
    y = y.double()
    cos, sin = cs.double().unsqueeze(1).chunk(2, -1)
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2).to(dt)
    a, b = y.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(dt)


def _plain_write(st):
    case, dt = st["case"], _io(st["case"])
    L, mode = case["latent"], case["mode"]
    cs = st["cos_sin"][st["positions"].long()]
    q = _rotated(st["q"][..., NOPE:], cs, case["interleaved"], dt)
    kr = _rotated(st["ckr"][:, None, L:], cs, case["interleaved"], dt)[:, 0]
    c = st["ckr"][:, :L].double()
    if st["w"] is not None:
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + 1e-6) * st["w"].double()
    c = c.to(dt)
    back = _value(*_quantize(c.float(), mode, _scale(mode)), mode, _scale(mode)).to(dt)
    return q, c, kr, back, kr.half().to(dt)


def _padded(st):
    """Rows of q by sequence, [B, max_q], which of them exist, and [B, max_q, S]: token s is seen by query i."""
    case, cu, n = st["case"], st["cu"].long(), st["seq_lens"].long()
    row = cu[:-1, None] + torch.arange(st["max_q"], device="cuda")
    real = row < cu[1:, None]
    s = torch.arange(st["max_n"], device="cuda")
    see = (s < n[:, None]).unsqueeze(1).expand(-1, st["max_q"], -1)
    if case["causal"]:
        m = cu[1:] - cu[:-1]
        see = see & (s <= ((n - m)[:, None] + torch.arange(st["max_q"], device="cuda")).unsqueeze(-1))
    return row.clamp(max=st["q"].shape[0] - 1), real, see


def _softmax(s, see, scale):
    """Weights, their sums and log-sum-exps of scores [.., S]."""
    s = (s * scale).masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    s = torch.exp(s - top)
    l = s.sum(-1, keepdim=True)
    return s, l.clamp_min(1e-30), (top + torch.log(l)).squeeze(-1)


def _plain_attend(st):
    case = st["case"]
    L, H, B, m = case["latent"], case["heads"], case["seqs"], st["max_q"]
    blk = st["pool"][256:].reshape(-1, P * _row_bytes(case["mode"], L))[st["table"].long()]
    c, kr = _unpack(blk, case["mode"], L, _scale(case["mode"]))  # [B, pages, P, ..]
    k = torch.cat([c, kr], -1).flatten(1, 2)[:, :st["max_n"]]
    row, real, see = _padded(st)
    s = (st["q"][row].float().reshape(B, m * H, L + ROPE) @ k.transpose(-1, -2)).reshape(B, m, H, -1)
    w, l, lse = _softmax(s, see.unsqueeze(2), st["scale"])
    o = ((w.reshape(B, m * H, -1) @ k[..., :L]).reshape(B, m, H, L) / l)[real].to(_io(case))
    return (o, lse[real]) if case["lse"] else o


def _plain_prompt(st):
    case = st["case"]
    row, real, see = _padded(st)
    at = st["cu_k"][:-1].long()[:, None] + torch.arange(st["max_n"], device="cuda")
    at = at.clamp(max=st["kv"].shape[0] - 1)  # (rows past a sequence's end are masked)
    kv = st["kv"][at].float().transpose(1, 2)  # [B, H, S, 2 NOPE]
    q = st["q"][row].float().transpose(1, 2)   # [B, H, m, NOPE + ROPE]
    s = q[..., :NOPE] @ kv[..., :NOPE].transpose(-1, -2) + q[..., NOPE:] @ st["kr"][at].float().transpose(-1, -2).unsqueeze(1)
    w, l, lse = _softmax(s, see.unsqueeze(1), st["scale"])
    o = (w @ kv[..., NOPE:] / l).transpose(1, 2)[real].to(_io(case))
    return (o, lse.transpose(1, 2)[real]) if case["lse"] else o


# ---------------------------------------------------------------- from the definition, in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    return {"read": _exact_read, "write": _exact_write, "attend": _exact_attend, "prompt": _exact_prompt}[case["op"]](case, st)


def _fp8(b):
    """E4M3 bytes -> fp64, from the format's definition."""
    b = b.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * 2.0 ** (e - 10).double())
    return torch.where(b >> 7 == 1, -mag, mag)


def _exact_rows(case, st, slots):
    """Latents [n, L] and rotary parts [n, ROPE] at `slots`, fp64, written from the layout byte by byte."""
    mode, L = case["mode"], case["latent"]
    base = 256 + (slots // P) * P * _row_bytes(mode, L)
    t = slots % P
    d, r = torch.arange(L, device="cuda"), torch.arange(ROPE, device="cuda")
    byte = lambda i: st["pool"][i].to(torch.int64)  # noqa: E731
    side = P * L // 2 if mode == "nvfp4" else P * L
    at = base + side + 2 * P * ROPE  # the scales
    h = (base + side + t * 2 * ROPE)[:, None] + 2 * r
    h = byte(h) | (byte(h + 1) << 8)
    e, m = (h >> 10) & 31, (h & 1023).double()
    rope = torch.where(e == 0, m * 2.0 ** -24, (1024.0 + m) * 2.0 ** (e - 25).double())
    rope = torch.where(h >> 15 == 1, -rope, rope)
    one = float(torch.tensor(_scale(mode), dtype=torch.float32))
    if mode == "nvfp4":
        c = byte((base + t * (L // 2))[:, None] + d // 2) >> (4 * (d % 2))
        mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[c & 7]
        s = _fp8(byte((at + t * (L // 16))[:, None] + d // 16)) * one
        return torch.where((c >> 3) & 1 == 1, -mag, mag) * s, rope
    c = byte((base + t * L)[:, None] + d)
    c = (c - 256 * (c >> 7)).double() if mode == "int8_per_token_head" else _fp8(c)
    if mode == "fp8_per_tensor":
        return c * one, rope
    w = sum(byte(at + 4 * t + j) << (8 * j) for j in range(4)).to(torch.int32).view(torch.float32).double()
    return c * w[:, None], rope


def _exact_read(case, st):
    parts = [_exact_rows(case, st, st["slots"][a:a + 4096].long()) for a in range(0, case["tokens"], 4096)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _exact_write(case, st):
    L, half = case["latent"], ROPE // 2
    ang = st["cos_sin"][st["positions"].long()].double()

    def turn(y):
        z = y.clone()
        for j in range(half):
            a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
            c, s = ang[:, j, None], ang[:, half + j, None]
            z[..., a] = y[..., a] * c - y[..., b] * s
            z[..., b] = y[..., a] * s + y[..., b] * c
        return z
    x = st["ckr"].double()
    c = x[:, :L]
    if st["w"] is not None:
        c = c / torch.sqrt(c.square().sum(-1, keepdim=True) / L + 1e-6) * st["w"].double()
    # codes are whole numbers of a coarse grid: what they stand for has no 64-bit value of its own
    return turn(st["q"][..., NOPE:].double()), c, turn(x[:, None, L:])[:, 0], None, None


def _exact_one(case, st, b, q0, q1, n, keys, values):
    """Outputs and log-sum-exps of one sequence's queries; keys(h), values(h): [n, ..] of head h."""
    H = case["heads"]
    out, lse = [], []
    tok = torch.arange(n, device="cuda")
    for h in range(H):
        k, v = keys(h), values(h)
        for a in range(q0, q1, 512):
            x = st["q"][a:min(a + 512, q1), h].double()
            s = torch.einsum("id,td->it", x, k) * st["scale"]
            if case["causal"]:
                s = s.masked_fill(tok > (n - (q1 - a) + torch.arange(x.shape[0], device="cuda"))[:, None], -math.inf)
            lse.append(torch.logsumexp(s, -1))
            out.append(torch.softmax(s, -1) @ v)
    m = q1 - q0
    return torch.cat(out).reshape(H, m, -1).transpose(0, 1), torch.cat(lse).reshape(H, m).t()


def _exact_all(case, st, rows):
    q, n = _lens(case)
    out, lse, at = [], [], 0
    for b in range(len(q)):
        if q[b]:
            o, x = _exact_one(case, st, b, at, at + q[b], n[b], *rows(b, n[b]))
            out.append(o)
            lse.append(x)
        at += q[b]
    return (torch.cat(out), torch.cat(lse)) if case["lse"] else torch.cat(out)


def _exact_attend(case, st):
    def rows(b, n):
        t = torch.arange(n, device="cuda")
        c, kr = _exact_rows(case, st, st["table"][b, t // P].long() * P + t % P)
        k = torch.cat([c, kr], -1)
        return (lambda h: k), (lambda h: c)
    return _exact_all(case, st, rows)


def _exact_prompt(case, st):
    starts = st["cu_k"].tolist()

    def rows(b, n):
        kv, kr = st["kv"][starts[b]:starts[b] + n], st["kr"][starts[b]:starts[b] + n].double()
        return (lambda h: torch.cat([kv[:, h, :NOPE].double(), kr], -1)), (lambda h: kv[:, h, NOPE:].double())
    return _exact_all(case, st, rows)

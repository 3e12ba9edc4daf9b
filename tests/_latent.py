"""Shared by the latent-cache tests: the page layout decoded byte by byte in
64 bits, caches filled through the library, and the formulas."""
from __future__ import annotations

import math

import torch

from _helpers import guarded, kvq

P, R = 16, 64
MODES = ["fp8_per_tensor", "int8_per_token_head", "fp8_per_token_head", "nvfp4", "nvfp4_4over6"]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def four(mode):
    return mode.startswith("nvfp4")


def row_bytes(mode, L):
    return 2 * R + (L // 2 + L // 16 if four(mode) else L if mode == "fp8_per_tensor" else L + 4)


def e4m3(b):
    b = b.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * 2.0 ** (e - 10).double())
    mag = torch.where((b & 127) == 127, float("nan"), mag)
    return torch.where(b >> 7 == 1, -mag, mag)


def decode(pool, mode, L, slots):
    """(latents [n][L], rotary parts [n][R]) fp64 of a pool's slots, from the layout (CPU)."""
    pool, slots = pool.cpu(), slots.cpu().long()
    st = pool[16:20].view(torch.float32).double()
    base, t = 256 + (slots // P) * P * row_bytes(mode, L), slots % P
    codes = P * (L // 2 if four(mode) else L)
    rope = torch.stack([pool[(base + codes + t * 2 * R)[:, None] + 2 * torch.arange(R) + i] for i in (0, 1)], -1)
    rope = rope.contiguous().view(torch.float16).squeeze(-1).double()
    at = base + codes + P * 2 * R
    d = torch.arange(L)
    if four(mode):
        c = (pool[(base + t * (L // 2))[:, None] + d // 2] >> (4 * (d % 2)).to(torch.uint8)).long()
        mag = torch.tensor(E2M1, dtype=torch.float64)[c & 7]
        v = torch.where((c >> 3) & 1 == 1, -mag, mag)
        return v * e4m3(pool[(at + t * (L // 16))[:, None] + d // 16]) * st, rope
    c = pool[(base + t * L)[:, None] + d]
    c = c.view(torch.int8).double() if mode.startswith("int8") else e4m3(c)
    if mode == "fp8_per_tensor":
        return c * st, rope
    s = torch.stack([pool[at + 4 * t + i] for i in range(4)], -1).contiguous().view(torch.float32).double()
    return c * s, rope


def empty_cache(mode, L, pages, io=torch.float16, scale=9.0):
    """A cache over a guarded pool; scale: the largest value that the per-tensor scale covers."""
    K = kvq()
    cfg = K.make_latent_config(pages, P, L, R, mode, io)
    cache = K.kvq_latent_alloc(cfg, guarded(K.kvq_latent_bytes(cfg), torch.uint8, fill=0xCD, name="pool"))
    if mode == "fp8_per_tensor" or four(mode):
        K.kvq_latent_set_scale(cache, scale / (448.0 if mode == "fp8_per_tensor" else 2688.0))
    return cache


def identity_table(n):
    """cos_sin that rotates nothing: [n][R]."""
    return torch.cat([torch.ones(n, R // 2), torch.zeros(n, R // 2)], 1).cuda()


class Batch:
    """Sequences of n[b] cached tokens whose last m[b] have queries, on scattered pages."""

    def __init__(self, mode, L, m, n, heads, io=torch.float16, seed=0, spread=None, q_size=0.6, extra_rows=0, bad_ids=-7):
        g = torch.Generator().manual_seed(seed)
        K = kvq()
        per = [(x + P - 1) // P for x in n]
        pages = sum(per) + 3
        perm = torch.randperm(pages, generator=g).int()
        self.table = torch.full((len(n), max(max(per), 1)), bad_ids, dtype=torch.int32)
        at = 0
        for b, x in enumerate(per):
            self.table[b, :x] = perm[at:at + x]
            at += x
        self.mode, self.L, self.m, self.n, self.heads, self.io = mode, L, m, n, heads, io
        self.cache = empty_cache(mode, L, pages, io)
        c, kr = torch.randn(sum(n), L, generator=g), 1.5 * torch.randn(sum(n), R, generator=g)
        if spread is not None:
            c = (c * torch.exp(spread * torch.randn(sum(n), 1, generator=g))).clamp(-60000, 60000)  # (finite in fp16)
        self.slots = torch.cat([self.table[b, torch.arange(x) // P] * P + torch.arange(x) % P for b, x in enumerate(n)]
                               + [torch.zeros(0, dtype=torch.int32)]).int()
        if sum(n):
            K.kvq_latent_write(self.cache, c.to(io).cuda(), kr.to(io).cuda(), torch.zeros(sum(n), dtype=torch.int32).cuda(),
                               identity_table(1), slot_mapping=self.slots.cuda())
        self.q = (q_size * torch.randn(sum(m) + extra_rows, heads, L + R, generator=g)).to(io)
        cu = [sum(m[:b]) for b in range(len(m) + 1)]
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.scale = 192.0 ** -0.5

    def run(self, out_dtype=None, causal=True, lse=True, max_q=None, max_n=None, cache=None, stream=None, q=None, check=0):
        K = kvq()
        q = (self.q if q is None else q).cuda()
        odt = out_dtype or self.io
        out = guarded((q.shape[0], self.heads, self.L), odt, fill=float("nan"), name="out")
        ls = guarded((q.shape[0], self.heads), torch.float32, fill=float("nan"), name="lse") if lse else None
        max_q, max_n = max_q or max(max(self.m), 1), max_n if max_n is not None else max(self.n)
        table = self.table
        if max_n > table.shape[1] * P:
            table = torch.nn.functional.pad(table, (0, (max_n + P - 1) // P - table.shape[1]), value=-7)
        self.splits, ws = K.kvq_latent_plan(self.cache, q.shape[0], len(self.n), self.heads, max_q_len=max_q, max_seq_len=max_n)
        work = guarded(max(ws, 16), torch.uint8, fill=0xFF, name="workspace")
        K.kvq_latent_attention(self.cache, q, self.cu.cuda(), table.cuda(), torch.tensor(self.n, dtype=torch.int32).cuda(), out,
                               max_q_len=max_q, max_seq_len=max_n, softmax_scale=self.scale, causal=causal, lse=ls,
                               workspace=work, stream=stream)
        torch.cuda.synchronize()
        assert K.kvq_latent_read_errors(self.cache) == check
        return out.cpu(), (ls.cpu() if lse else None)

    def unit(self, b):
        """What a code of 1 stands for, token by token: [n][1] fp64."""
        st = self.cache.pool[16:20].cpu().view(torch.float32).double()
        s = self.slots[sum(self.n[:b]):sum(self.n[:b + 1])].long()
        if not self.mode.endswith("per_token_head"):
            return st.expand(len(s), 1)
        at = 256 + s // P * P * row_bytes(self.mode, self.L) + P * (self.L + 2 * R) + 4 * (s % P)
        return self.cache.pool.cpu()[at[:, None] + torch.arange(4)].contiguous().view(torch.float32).double()

    def keys(self, b):
        s = self.slots[sum(self.n[:b]):sum(self.n[:b + 1])]
        return decode(self.cache.pool, self.mode, self.L, s)

    def reference(self, causal=True, q=None, drop=()):
        """(out, lse, tolerance of out, tolerance of lse) in 64 bits; drop: (sequence, page) pairs that are missing.

        Tolerances.  Scores are sums of exact products (an fp16 query times exact codes), summed in fp32 by (L + R) / 16
        steps that may each cut off 2^-23 of the magnitudes' sum, and rounded a few times more: d = (steps + 4) 2^-23 of
        scale sum |q k| of a score.  A weight is then off by 2 d (score and log-sum-exp) and 2^-22 of the exponential; in the
        tensor-core path by fp16's half step 2^-11 too, and its sums over tokens by 2^-23 a step of 16 tokens.  Fp32 paths
        round every term of a score and of a sum: L + R and n steps of 2^-24.
        An fp16 weight is 2^(y - M) u_t of a token's unit u_t, off by half a step, 2^-11 of it, or 2^-25 where that is more;
        2^M is at most 2^-5 of the largest 2^y u (M = ceil(largest y + floor(log2 u)) - 6, or less).  Times the token's codes
        c_t / u_t, over all tokens and with weights w: 2^-30 max(w u) sum |c_t| / u_t."""
        q = (self.q if q is None else q).double()
        out, lse, tol, ltol = [], [], [], []
        for b in range(len(self.m)):
            c, kr = self.keys(b)
            k = torch.cat([c, kr], 1)
            n, m = self.n[b], self.m[b]
            x = q[int(self.cu[b]):int(self.cu[b]) + m]
            s = torch.einsum("ihd,td->iht", x, k) * self.scale
            pos = torch.arange(n - m, n) if causal else torch.full((m,), n - 1)
            see = torch.arange(n) <= pos[:, None, None]
            for bb, page in drop:
                if bb == b:
                    see = see & (torch.arange(n) // P != page)
            see = see.expand_as(s)
            s = s.masked_fill(~see, -math.inf)
            ls = torch.logsumexp(s, -1) if n else torch.full(s.shape[:2], -math.inf, dtype=torch.float64)
            w = torch.where(see, torch.exp(s - torch.where(ls == -math.inf, 0.0, ls).unsqueeze(-1)), 0.0)
            out.append(torch.einsum("iht,td->ihd", w, c))
            lse.append(ls)
            size = torch.einsum("ihd,td->iht", x.abs(), k.abs()) * self.scale
            size = torch.where(see, size, 0.0).amax(-1) if n else torch.zeros(s.shape[:2], dtype=torch.float64)
            exact = self.io == torch.float16
            d = ((self.L + R) / 16 + 4 if exact else self.L + R + 4) * 2.0 ** (-23 if exact else -24) * size
            mass = torch.einsum("iht,td->ihd", w, c.abs())
            u = self.unit(b)
            small = 2.0 ** -30 * (w * u[:, 0]).amax(-1, keepdim=True) * (c.abs() / u).sum(0) if n else 0.0 * mass
            steps = n / 16 * 2.0 ** -23 if exact else (n + 8) * 2.0 ** -24
            tol.append((mass, mass * (2 * d.unsqueeze(-1) + 2.0 ** -21 + steps) + (small if exact else 0.0)))
            ltol.append(d + 2.0 ** -21 + 2.0 ** -22 * torch.where(ls == -math.inf, 0.0, ls).abs())
        self.mass = torch.cat([t[0] for t in tol])
        return torch.cat(out), torch.cat(lse), torch.cat([t[1] for t in tol]), torch.cat(ltol)


def compare(got, ref, tol, weights_f16):
    """|got - ref| <= tol + the outputs' own rounding (+ half a step of fp16 weights, given as their mass)."""
    half = torch.finfo(got.dtype).eps / 2
    bound = tol * (1 + half) + half * ref.abs() + (2.0 ** -25 if got.dtype == torch.float16 else 1e-30)
    if weights_f16 is not None:
        bound = bound + 2.0 ** -11 * weights_f16
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all()), "non-finite output"
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.2f} of its bound"
    return worst

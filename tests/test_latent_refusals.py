"""Refusals of the latent calls: every bad argument is an error before anything
is launched (no GPU needed: the buffers are never touched)."""
import ctypes

import pytest

from _helpers import kvq

INVALID, UNSUPPORTED, MISMATCH, CAPACITY = 1, 2, 3, 4


def _config(**kw):
    c = dict(num_pages=4, page_size=16, latent_dim=512, rope_dim=64, mode="fp8_per_token_head", io_dtype=0)
    c.update(kw)
    return kvq().make_latent_config(**c)


@pytest.mark.parametrize("kw,status", [
    (dict(num_pages=0), INVALID), (dict(num_pages=1 << 28), UNSUPPORTED), (dict(page_size=128), UNSUPPORTED),
    (dict(latent_dim=128), UNSUPPORTED), (dict(latent_dim=0), UNSUPPORTED), (dict(rope_dim=32), UNSUPPORTED),
    (dict(mode="int4_per_token_head"), UNSUPPORTED), (dict(mode="kvarn_k4v2_g128"), UNSUPPORTED), (dict(mode=0), UNSUPPORTED)])
def test_config(kw, status):
    K = kvq()
    with pytest.raises(K.KVQError) as e:
        K.kvq_latent_bytes(_config(**kw))
    assert e.value.status == status


@pytest.mark.parametrize("mode,page", [("fp8_per_tensor", 16 * 640), ("int8_per_token_head", 16 * 644),
                                       ("fp8_per_token_head", 16 * 644), ("nvfp4", 16 * 416), ("nvfp4_4over6", 16 * 416)])
def test_sizes(mode, page):
    assert kvq().kvq_latent_bytes(_config(mode=mode)) == 256 + 4 * page


class _Handle(ctypes.Structure):
    """The start of the library's descriptor: its config (the calls below read no more before they refuse)."""
    _fields_ = [("cfg", kvq().LatentConfig), ("base", ctypes.c_void_p), ("page_bytes", ctypes.c_size_t)]


@pytest.fixture
def handle():
    return _Handle(_config(), 0x100000, 16 * 644)


def status(rc):
    return rc


def _attend(h, **kw):
    K = kvq()
    a = dict(q=0x1000, total_q=4, cu=0x1000, table=0x1000, max_pages=4, lens=0x1000, seqs=2, heads=8, max_q=2, max_n=64, mode=3,
             scale=0.1, causal=1, out=0x1000, out_dtype=0, lse=None, ws=0x1000, ws_bytes=1 << 30)
    a.update(kw)
    return K.lib().kvq_latent_attention(None if h is None else ctypes.byref(h), a["q"], a["total_q"], a["cu"], a["table"], a["max_pages"],
                                        a["lens"], a["seqs"], a["heads"], a["max_q"], a["max_n"], a["mode"], a["scale"], a["causal"],
                                        a["out"], a["out_dtype"], a["lse"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(total_q=-1), INVALID), (dict(seqs=-1), INVALID), (dict(max_q=-1), INVALID), (dict(max_n=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(heads=0), INVALID), (dict(heads=70000), UNSUPPORTED), (dict(max_n=65), INVALID),
    (dict(total_q=2 ** 30, heads=8), UNSUPPORTED), (dict(mode=2), MISMATCH), (dict(out_dtype=2), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(max_q=0), INVALID),
    (dict(q=None), INVALID), (dict(q=0x1008), INVALID), (dict(out=None), INVALID), (dict(out=0x1004), INVALID), (dict(cu=None), INVALID),
    (dict(cu=0x1002), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(lens=0x1001), INVALID),
    (dict(lse=0x1002), INVALID), (dict(max_pages=6000, max_n=90000, ws=None), CAPACITY),
    (dict(max_pages=6000, max_n=90000, ws_bytes=64), CAPACITY), (dict(max_pages=6000, max_n=90000, ws=0x1008), INVALID)])
def test_attention(handle, kw, want):
    assert _attend(handle, **kw) == want
    assert kvq().lib().kvq_last_error()


def test_attention_nothing_to_do(handle):
    assert _attend(None) == INVALID
    assert _attend(handle, total_q=0, q=None, out=None) == 0
    assert _attend(handle, seqs=0, q=None, out=None) == 0


def _write(h, **kw):
    K = kvq()
    a = dict(latent=0x1000, k_rope=0x1000, q_rope=0x1000, q_rope_out=0x1000, latent_stride=512, k_rope_stride=64, q_stride=512,
             q_head_stride=64, q_out_stride=512, q_out_head_stride=64, latent_weight=None, positions=0x1000, cos_sin=0x1000,
             slot_mapping=0x1000, latent_out=None, k_rope_out=None, num_tokens=3, num_q_heads=8, max_position=16, interleaved=0,
             eps=1e-6)
    mode = kw.pop("mode", 3)
    a.update(kw)
    return K.lib().kvq_latent_write(ctypes.byref(h), ctypes.byref(K.LatentRows(**a)), mode, None)


@pytest.mark.parametrize("kw,want", [
    (dict(mode=2), MISMATCH), (dict(num_tokens=-1), INVALID), (dict(max_position=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(q_rope=None), INVALID), (dict(q_rope_out=None), INVALID), (dict(num_q_heads=0), INVALID),
    (dict(latent_stride=516), INVALID), (dict(q_head_stride=-64), INVALID), (dict(q_out_stride=4), INVALID),
    (dict(latent=None), INVALID), (dict(latent=0x1008), INVALID), (dict(k_rope=None), INVALID), (dict(positions=None), INVALID),
    (dict(cos_sin=0x1008), INVALID), (dict(slot_mapping=0x1002), INVALID), (dict(latent_out=0x1008), INVALID)])
def test_write(handle, kw, want):
    assert _write(handle, **kw) == want
    assert kvq().lib().kvq_latent_write(ctypes.byref(handle), None, 3, None) == INVALID


def test_read_and_scale(handle):
    L, h = kvq().lib(), ctypes.byref(handle)
    assert L.kvq_latent_read(h, 0x1000, -1, 0x1000, None, 0, None) == INVALID
    assert L.kvq_latent_read(h, 0x1000, 1, 0x1000, None, 5, None) == UNSUPPORTED
    assert L.kvq_latent_read(h, None, 1, 0x1000, None, 0, None) == INVALID
    assert L.kvq_latent_read(h, 0x1000, 1, 0x1008, None, 0, None) == INVALID
    assert L.kvq_latent_read(h, None, 0, None, None, 0, None) == 0
    assert L.kvq_latent_set_scale(h, 0.0, None) == INVALID
    assert L.kvq_latent_set_scale(h, float("inf"), None) == INVALID
    assert L.kvq_latent_set_scale_from_amax(h, 0x1000, None) == MISMATCH  # the mode has scales of its own
    assert L.kvq_latent_set_scale_from_amax(h, None, None) == INVALID
    assert L.kvq_latent_alloc(ctypes.byref(_config()), 0x1010, 1 << 30, ctypes.byref(ctypes.c_void_p())) == INVALID
    assert L.kvq_latent_alloc(ctypes.byref(_config()), 0x1000, 300, ctypes.byref(ctypes.c_void_p())) == CAPACITY
    assert L.kvq_latent_free(None) == 0


def _prompt(h, **kw):
    K = kvq()
    a = dict(q=0x1000, k=0x1000, k_rope=0x1000, v=0x1000, k_stride=2048, k_head_stride=256, v_stride=2048, v_head_stride=256,
             k_rope_stride=64, cu_q_lens=0x1000, cu_k_lens=0x1000, out=0x1000, lse=None, total_q=4, total_k=9, num_seqs=2, num_q_heads=8,
             max_q_len=2, max_k_len=5, causal=1, out_dtype=0, softmax_scale=0.1)
    a.update(kw)
    return K.lib().kvq_latent_prompt_attention(ctypes.byref(h), ctypes.byref(K.LatentPrompt(**a)), None)


@pytest.mark.parametrize("kw,want", [
    (dict(total_q=-1), INVALID), (dict(total_k=-1), INVALID), (dict(num_seqs=-1), INVALID), (dict(num_q_heads=0), INVALID),
    (dict(max_q_len=0), INVALID), (dict(max_k_len=-1), INVALID), (dict(out_dtype=9), UNSUPPORTED), (dict(softmax_scale=-1.0), INVALID),
    (dict(k_stride=2050), INVALID), (dict(v_head_stride=-256), INVALID), (dict(k_rope_stride=68), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=0x1008), INVALID), (dict(k_rope=0x1008), INVALID), (dict(cu_q_lens=None), INVALID),
    (dict(cu_k_lens=None), INVALID), (dict(cu_k_lens=0x1002), INVALID), (dict(out=0x1008), INVALID), (dict(lse=0x1001), INVALID)])
def test_prompt(handle, kw, want):
    assert _prompt(handle, **kw) == want


def test_prompt_nothing_to_do(handle):
    assert _prompt(handle, total_q=0, q=None) == 0
    assert _prompt(handle, num_seqs=0, q=None) == 0


def test_the_other_calls_do_not_take_a_latent_cache():
    K = kvq()
    assert not hasattr(K.LatentCache, "handle")

"""Refusals of the serving calls on the host: parameters, pointers, workspaces (no kernel runs), and the Python
wrappers' checks of tensors."""
import ctypes

import pytest
import torch

from sparse_rank_attention_block_b200 import build, sda


@pytest.fixture(scope="module")
def L():
    build.build()
    return sda.lib()


def prompt(**kw):
    return sda.prompt_params(**{**dict(n_seq=2, rows_q=10, rows_k=10, H=4, H_kv=2, d=64), **kw})


def cache(**kw):
    return sda.cache_params(**{**dict(B=2, H=4, H_kv=2, d=64, block=16, n_blocks=8, max_blocks=4, rows=2, max_new=1,
                                      keep=16, recent=4), **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=0), -3), (dict(n_seq=65536), -3), (dict(rows_q=0), -3), (dict(rows_k=0), -3), (dict(H_kv=3), -3),
    (dict(H_kv=0), -3), (dict(H=0), -3), (dict(H=2048, H_kv=1), -4), (dict(d=96), -4), (dict(causal=2), -3),
    (dict(ld_q=255), -3), (dict(ld_q=260), -2), (dict(ld_k=120), -3), (dict(ld_v=132), -2), (dict(ld_o=1 << 33), -4),
    (dict(scale=-1.0), -3), (dict(scale=float("nan")), -3), (dict(scale=float("inf")), -3), (dict(scale=1e-60), -3),
    (dict(rows_q=(1 << 30) + 1), -4)])
def test_prompt_params_refused(L, kw, code):
    p = prompt()
    for n, v in kw.items():
        setattr(p, n, v)
    assert L.sda_prompt_workspace_size(ctypes.byref(p)) == 0
    assert L.sda_prompt_attn_fwd(ctypes.byref(p), *([16] * 7), 256, 1 << 20, None) == code
    assert L.sda_last_error_detail()


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), -3), (dict(B=65536), -3), (dict(H_kv=3), -3), (dict(d=80), -4), (dict(block=8), -4),
    (dict(block=48), -4), (dict(block=256), -4), (dict(n_blocks=0), -3), (dict(max_blocks=0), -3), (dict(rows=-1), -3),
    (dict(max_new=-1), -3), (dict(keep=-1), -3), (dict(recent=-1), -3), (dict(recent=17), -3), (dict(weights=2), -3),
    (dict(ld_q=264 + 4), -2), (dict(ld_k=64), -3), (dict(scale=-0.5), -3), (dict(n_blocks=1 << 27), -4),
    (dict(max_blocks=(1 << 20) + 1), -4), (dict(max_new=(1 << 20) + 1), -4)])
def test_cache_params_refused(L, kw, code):
    p = cache()
    for n, v in kw.items():
        setattr(p, n, v)
    b = ctypes.byref(p)
    assert L.sda_cache_workspace_size(b) == 0
    assert L.sda_cache_append(b, *([16] * 10), 256, 1 << 30, None) == code
    assert L.sda_cache_attn_fwd(b, *([16] * 8), None, None, 16, 256, 1 << 30, None) == code
    assert L.sda_cache_evict(b, *([16] * 10), 256, 1 << 30, None) == code


def test_pointers_and_workspaces(L):
    p, c = prompt(), cache()
    n = L.sda_cache_workspace_size(ctypes.byref(c))
    assert L.sda_prompt_workspace_size(ctypes.byref(p)) == 256 and n >= 256
    calls = [(L.sda_prompt_attn_fwd, p, 7, 256, (6,)), (L.sda_cache_append, c, 10, 256, (9,)),
             (L.sda_cache_attn_fwd, c, 11, n, (8, 9)), (L.sda_cache_evict, c, 10, 256 + 2 * 2 * 16 * 4, ())]
    for fn, par, count, need, optional in calls:
        good = [None if i in optional else 16 for i in range(count)]
        b = ctypes.byref(par)
        assert fn(b, *good, 256, need - 1, None) == -5
        assert fn(b, *good, 128, need, None) == -2
        assert fn(b, *good, None, need, None) == -1
        assert fn(None, *good, 256, need, None) == -1
        for i in range(count):
            if i not in optional:
                assert fn(b, *[None if j == i else x for j, x in enumerate(good)], 256, need, None) == -1, (fn, i)
            if not (fn is L.sda_cache_attn_fwd and i in optional):
                assert fn(b, *[24 if j == i else x for j, x in enumerate(good)], 256, need, None) == -2, (fn, i)
        # everything in order: the next check is the device, which a host without a GPU does not have
        if not torch.cuda.is_available():
            assert fn(b, *good, 256, need, None) == -8


def test_rows_and_weights_needed(L):
    c = cache(max_new=0)
    assert L.sda_cache_append(ctypes.byref(c), *([16] * 10), 256, 1 << 30, None) == -3
    assert L.sda_cache_attn_fwd(ctypes.byref(c), *([16] * 8), None, None, 16, 256, 1 << 30, None) == -3
    c = cache()                                    # weights = 0
    assert L.sda_cache_attn_fwd(ctypes.byref(c), *([16] * 8), None, 16, 16, 256, 1 << 30, None) == -3
    assert b"weights" in L.sda_last_error_detail()
    c = cache(weights=True)                        # w_in without w_out
    assert L.sda_cache_attn_fwd(ctypes.byref(c), *([16] * 8), 16, None, 16, 256, 1 << 30, None) == -1
    c = cache(keep=0, recent=0)
    assert L.sda_cache_evict(ctypes.byref(c), *([16] * 10), 256, 1 << 30, None) == -3


def test_workspace_of_the_cache(L):
    """Weights cost the scores; partial outputs are those of one wave of CTAs, however many rows there are."""
    size = lambda **kw: L.sda_cache_workspace_size(ctypes.byref(cache(**kw)))  # noqa: E731
    big = dict(B=4, max_blocks=256, n_blocks=1024)
    assert size(**big, weights=True) >= size(**big) + 4 * 2 * 256 * 16 * 4 * 4
    assert size(B=64, H=32, H_kv=8, d=128, block=64, n_blocks=9216, max_blocks=144, rows=9216, max_new=9216) < 8 << 20


def _tensors():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(q=bf(10, 4, 64), k=bf(10, 2, 64), v=bf(10, 2, 64), seq_q=i32(3), seq_k=i32(3), o=bf(10, 4, 64),
                lse=torch.zeros(10, 4))


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(10, 4, 64)), ("q", torch.zeros(9, 4, 64, dtype=torch.bfloat16)),
    ("q", torch.zeros(10, 4, 128, dtype=torch.bfloat16)[:, :, ::2]),
    ("k", torch.zeros(10, 6, 64, dtype=torch.bfloat16)[:, :2]),          # rows apart, ld_k = 0
    ("v", torch.zeros(10, 2, 64, dtype=torch.float16)), ("seq_q", torch.zeros(3, dtype=torch.int64)),
    ("seq_k", torch.zeros(2, dtype=torch.int32)), ("o", torch.zeros(10, 4, 64)), ("lse", torch.zeros(10, 3)),
    ("lse", torch.zeros(10, 4, dtype=torch.float64))])
def test_wrapper_refuses_tensors(L, name, bad):
    t = _tensors()
    t[name] = bad
    with pytest.raises(sda.SdaError) as e:
        sda.sda_prompt_attn_fwd(prompt(), *t.values(), 256, 256, stream=0)
    assert e.value.code == -3 and name in str(e.value)


def test_wrapper_takes_rows_apart_and_refuses_host_tensors(L):
    t = _tensors()
    wide = torch.zeros(10, 8, 64, dtype=torch.bfloat16)
    t["q"], t["k"], t["v"] = wide[:, :4], wide[:, 4:6], wide[:, 6:]
    with pytest.raises(sda.SdaError) as e:       # the layout passes, the place does not
        sda.sda_prompt_attn_fwd(prompt(ld_q=512, ld_k=512, ld_v=512), *t.values(), 256, 256, stream=0)
    assert e.value.code == -8


def test_cache_wrappers_refuse_tensors(L):
    c = cache(weights=True)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    codes, scale, w = torch.zeros(8, 2, 16, 64, dtype=torch.uint8), torch.zeros(8, 2), torch.zeros(8, 2, 16)
    pool = [i32(2), i32(2, 4), codes, codes.clone(), scale, scale.clone()]
    calls = [(sda.sda_cache_append, [bf(2, 2, 64), bf(2, 2, 64), i32(3), *pool, w]),
             (sda.sda_cache_attn_fwd, [bf(2, 4, 64), i32(3), *pool, w, w, bf(2, 4, 64)]),
             (sda.sda_cache_evict, [*pool, w, i32(2, 1), i32(2, 2, 16), i32(2)])]
    for fn, args in calls:
        with pytest.raises(sda.SdaError) as e:
            fn(c, *args, 256, 1 << 30, stream=0)
        assert e.value.code == -8
        for i, a in enumerate(args):
            for wrong in (a.to(torch.float64), a.flatten()[:-1].contiguous()):
                with pytest.raises(sda.SdaError) as e:
                    fn(c, *args[:i], wrong, *args[i + 1:], 256, 1 << 30, stream=0)
                assert e.value.code == -3, (fn.__name__, i)


def _cache_calls():
    """Each cache call's wrapper with host tensors of the right types and shapes, for cache(weights=True)."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    codes, scale, w = torch.zeros(8, 2, 16, 64, dtype=torch.uint8), torch.zeros(8, 2), torch.zeros(8, 2, 16)
    pool = [i32(2), i32(2, 4), codes, codes.clone(), scale, scale.clone()]
    return [(sda.sda_cache_append, [bf(2, 2, 64), bf(2, 2, 64), i32(3), *pool, w]),
            (sda.sda_cache_attn_fwd, [bf(2, 4, 64), i32(3), *pool, w, w, bf(2, 4, 64)]),
            (sda.sda_cache_evict, [*pool, w, i32(2, 1), i32(2, 2, 16), i32(2)])]


def test_wrappers_refuse_the_same_bytes_in_another_order(L):
    """Codes as [n_blocks, block, H_kv, d], scales by head, a table by column, lse by head: as many bytes, other
    meaning. A flat tensor says nothing about the order and is taken."""
    t = _tensors()
    t["lse"] = torch.zeros(4, 10)
    with pytest.raises(sda.SdaError) as e:
        sda.sda_prompt_attn_fwd(prompt(), *t.values(), 256, 256, stream=0)
    assert e.value.code == -3 and "lse" in str(e.value)
    for fn, args in _cache_calls():
        for i, a in enumerate(args):
            if a.dim() < 2 or a.dtype is torch.bfloat16 or a.shape[0] == a.shape[1]:
                continue                                   # equal extents: nothing tells the orders apart
            with pytest.raises(sda.SdaError) as e:
                fn(cache(weights=True), *args[:i], a.transpose(0, 1).contiguous(), *args[i + 1:], 256, 1 << 30, stream=0)
            assert e.value.code == -3, (fn.__name__, i)
            with pytest.raises(sda.SdaError) as e:         # the layout passes, the place does not
                fn(cache(weights=True), *args[:i], a.flatten(), *args[i + 1:], 256, 1 << 30, stream=0)
            assert e.value.code == -8, (fn.__name__, i)
        swapped = [a.transpose(1, 2).contiguous() if a.dim() == 4 else a for a in args]
        with pytest.raises(sda.SdaError) as e:
            fn(cache(weights=True), *swapped, 256, 1 << 30, stream=0)
        assert e.value.code == -3 and "k_codes" in str(e.value)


def test_wrappers_take_codes_in_torchs_own_type(L):
    for fn, args in _cache_calls():
        for kind, code in ((torch.float8_e4m3fn, -8), (torch.float8_e5m2, -3), (torch.int8, -3)):  # -8: the layout passes
            typed = [a.view(kind) if a.dtype is torch.uint8 else a for a in args]
            with pytest.raises(sda.SdaError) as e:
                fn(cache(weights=True), *typed, 256, 1 << 30, stream=0)
            assert e.value.code == code, (fn.__name__, kind)

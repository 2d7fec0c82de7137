"""GPU parity of the serving operators against the fp64 oracle, at the sizes and masks where they can go wrong.

Bars: attention within attention_tolerance (derived in _serving.py); codes, scales, kept positions and moved
weights exactly; collected weights within their fp32 bound. Everything outside the sequences holds NaN or a mark
that has to be there afterwards.
"""
import numpy as np
import pytest
import torch

import oracle.serving as O
from sparse_rank_attention_block_b200 import sda

from _gpu import ensure_lib
from _serving import (U_BF16, U_F16, U_F32, attention_tolerance, bf16, f64, make_pool, make_table, offsets, score_size)

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


# --------------------------------------------------------------------------------------------- prompt attention

def run_prompt(q, k, v, sq, sk, causal, scale=0.0, ld=None, stream=None, lse=True):
    """q, k, v on the device, [rows, heads, d] views; returns o, lse, both filled with marks before the call."""
    T, H, d = q.shape
    p = sda.prompt_params(n_seq=len(sq) - 1, rows_q=T, rows_k=k.shape[0], H=H, H_kv=k.shape[1], d=d, causal=causal,
                          scale=scale, **(ld or {}))
    ws = sda.Workspace(p)
    o = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    ls = torch.full((T, H), 7.0, device=DEV) if lse else None
    sda.sda_prompt_attn_fwd(p, q, k, v, dev(sq), dev(sk), o, ls, ws.ptr, ws.nbytes, stream)
    ws.check()
    return o, ls


def check_prompt(q, k, v, sq, sk, causal, o, lse, scale=None):
    want, want_lse, spread = O.prompt_attention(f64(q), f64(k), f64(v), sq, sk, causal, scale)
    got, got_lse = f64(o), f64(lse)
    inside = np.zeros(len(got), bool)
    for a, b in zip(sq[:-1], sq[1:]):
        inside[a:b] = True
    assert np.all(got[~inside] == 7) and np.all(got_lse[~inside] == 7), "rows outside the sequences were written"
    size = score_size(f64(q)[inside], f64(k)[sk[0]:sk[-1]], scale) if sk[-1] > sk[0] else 0.0
    tol = attention_tolerance(want[inside], spread[inside], size, q.shape[2], U_BF16)
    err = np.abs(got[inside] - want[inside])
    assert np.all(err <= tol), f"o: {np.max(err - tol):.3e} over the bound, worst error {err.max():.3e}"
    none = np.isneginf(want_lse[inside])
    assert np.array_equal(np.isneginf(got_lse[inside]), none)
    d_lse = np.abs(got_lse[inside] - want_lse[inside])[~none]
    bound = 2 * (q.shape[2] + 8) * U_F32 * size + 2.0 ** -18 * (1 + np.abs(want_lse[inside])[~none])
    assert np.all(d_lse <= bound), f"lse: worst error {d_lse.max():.3e}"


PROMPTS = [
    # n_q, n_k, H, H_kv, d, causal
    ([1], [1], 1, 1, 64, True),
    ([1], [1], 2, 1, 128, True),
    ([128], [128], 4, 2, 128, True),
    ([129], [129], 4, 1, 128, True),              # one row in the second tile
    ([127, 1, 0, 130], [127, 1, 0, 130], 6, 2, 64, True),   # heads odd in number per key head, an empty sequence
    ([300], [300], 3, 3, 128, True),              # two row tiles of one head, the last partial
    ([257], [257], 5, 1, 64, False),
    ([40, 200], [300, 5], 4, 2, 128, True),       # a later chunk; more queries than keys (rows that see nothing)
    ([40, 200], [300, 5], 2, 2, 64, True),
    ([3, 140], [0, 77], 4, 4, 128, True),         # no keys at all
    ([3, 140], [0, 77], 4, 2, 128, False),
    ([700, 33, 64, 256], [700, 33, 64, 256], 4, 2, 64, True),
    ([260], [1031], 4, 2, 128, False),            # more K and V tiles than the ring holds
]


@pytest.mark.parametrize("nq,nk,H,H_kv,d,causal", PROMPTS)
def test_prompt(nq, nk, H, H_kv, d, causal):
    rng = np.random.default_rng(sum(nq) + 7 * H + d)
    lead, behind = 3, 5                           # rows of nobody around the sequences, NaN and infinity
    sq, sk = offsets(nq, lead), offsets(nk, lead)
    q, k, v = (bf16((lead + sum(n) + behind, h, d), rng) for n, h in ((nq, H), (nk, H_kv), (nk, H_kv)))
    for x, a in ((q, sq), (k, sk), (v, sk)):
        x[:lead], x[a[-1]:] = float("nan"), float("inf")
    q, k, v = q.to(DEV), k.to(DEV), v.to(DEV)
    o, lse = run_prompt(q, k, v, sq, sk, causal)
    check_prompt(q, k, v, sq, sk, causal, o, lse)
    again, lse2 = run_prompt(q, k, v, sq, sk, causal)
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    bare, _ = run_prompt(q, k, v, sq, sk, causal, lse=False)
    assert torch.equal(o, bare)


def test_prompt_many_sequences():
    """More sequences than a warp has lanes, among them empty ones."""
    rng = np.random.default_rng(5)
    n = [int(x) for x in rng.integers(0, 150, 71)]
    sq = offsets(n)
    q, k, v = (bf16((sq[-1], h, 64), rng).to(DEV) for h in (2, 1, 1))
    o, lse = run_prompt(q, k, v, sq, sq, True)
    check_prompt(q, k, v, sq, sq, True, o, lse)


@pytest.mark.parametrize("H,H_kv,d,causal", [(16, 8, 128, True), (8, 8, 64, True), (16, 8, 64, False), (8, 8, 128, False)])
def test_prompt_several_tiles_for_each_cta(H, H_kv, d, causal):
    """Far more tiles than SMs, of unequal lengths, among them tiles without a visible key and sequences without
    rows or keys: every CTA goes from one to the next."""
    rng = np.random.default_rng(22)
    nq = [int(x) for x in rng.integers(0, 60, 70)] + [300, 0, 140, 1]
    nk = [int(x) for x in rng.integers(0, 60, 70)] + [310, 40, 10, 700]
    sq, sk = offsets(nq), offsets(nk)
    q, k, v = (bf16((int(a[-1]), h, d), rng).to(DEV) for a, h in ((sq, H), (sk, H_kv), (sk, H_kv)))
    o, lse = run_prompt(q, k, v, sq, sk, causal)
    check_prompt(q, k, v, sq, sk, causal, o, lse)
    for _ in range(3):
        again, lse2 = run_prompt(q, k, v, sq, sk, causal)
        assert torch.equal(o, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("scale", [0.5, 0.003])
def test_prompt_scale_and_slices_of_one_projection(scale):
    rng = np.random.default_rng(6)
    H, H_kv, d, n = 4, 2, 128, [150, 90]
    rows = bf16((240, (H + 2 * H_kv) * d), rng).to(DEV)
    q, k, v = (x.unflatten(1, (h, d)) for x, h in zip(rows.split([H * d, H_kv * d, H_kv * d], 1), (H, H_kv, H_kv)))
    ld = rows.shape[1]
    sq = offsets(n)
    o, lse = run_prompt(q, k, v, sq, sq, True, scale, dict(ld_q=ld, ld_k=ld, ld_v=ld))
    check_prompt(q, k, v, sq, sq, True, o, lse, scale)


def test_prompt_growing_maximum():
    """Scores that grow by far more than 2^8 from key tile to key tile: the running reference moves."""
    rng = np.random.default_rng(7)
    n, d = 520, 64
    q, k, v = bf16((n, 2, d), rng), bf16((n, 1, d), rng), bf16((n, 1, d), rng)
    q[:, 0], q[:, 1] = 1.0, -1.0                 # one head sees the largest scores last, the other first
    k += (torch.arange(n) / 40.0).to(torch.bfloat16)[:, None, None]
    q, k, v = q.to(DEV), k.to(DEV), v.to(DEV)
    sq = offsets([n])
    for causal in (True, False):
        o, lse = run_prompt(q, k, v, sq, sq, causal)
        check_prompt(q, k, v, sq, sq, causal, o, lse)


def test_prompt_hidden_keys_of_the_sequence_do_not_change_a_row():
    """Causality: rewriting later tokens leaves the earlier rows bit for bit."""
    rng = np.random.default_rng(8)
    n, d = 400, 128
    q, k, v = (bf16((n, h, d), rng).to(DEV) for h in (4, 2, 2))
    sq = offsets([n])
    o, _ = run_prompt(q, k, v, sq, sq, True)
    for cut in (128, 200, 399):
        k2, v2 = k.clone(), v.clone()
        k2[cut:], v2[cut:] = 3.0, -5.0
        o2, _ = run_prompt(q, k2, v2, sq, sq, True)
        assert torch.equal(o[:cut], o2[:cut]) and not torch.equal(o[cut:], o2[cut:])


def test_prompt_bad_offsets_are_reported_and_stay_in_range():
    rng = np.random.default_rng(9)
    q, k, v = (bf16((64, h, 64), rng).to(DEV) for h in (2, 1, 1))
    for bad in ([0, 65], [-1, 64], [10, 5], [0, 1 << 30], [-(1 << 31), (1 << 31) - 1]):
        for which in range(2):
            p = sda.prompt_params(n_seq=1, rows_q=64, rows_k=64, H=2, H_kv=1, d=64)
            ws = sda.Workspace(p)
            o = torch.empty_like(q)
            s = [dev(np.array([0, 64], np.int32))] * 2
            s[which] = dev(np.array(bad, np.int64).astype(np.int32))
            sda.sda_prompt_attn_fwd(p, q, k, v, *s, o, None, ws.ptr, ws.nbytes)
            with pytest.raises(sda.SdaError) as e:
                ws.check()
            assert e.value.code == -3
            ws.check()                            # the read cleared the word


def test_prompt_captured_and_on_another_stream():
    """Captured once, replayed with other offsets and values in the same tensors; run on a side stream."""
    rng = np.random.default_rng(10)
    q, k, v = (bf16((300, h, 128), rng).to(DEV) for h in (4, 2, 2))
    p = sda.prompt_params(n_seq=2, rows_q=300, rows_k=300, H=4, H_kv=2, d=128)
    ws = sda.Workspace(p)
    o = torch.full_like(q, 7.0)
    lse = torch.full((300, 4), 7.0, device=DEV)
    seq = dev(offsets([100, 180]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sda.sda_prompt_attn_fwd(p, q, k, v, seq, seq, o, lse, ws.ptr, ws.nbytes)
    side.synchronize()
    check_prompt(q, k, v, offsets([100, 180]), offsets([100, 180]), True, o, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sda.sda_prompt_attn_fwd(p, q, k, v, seq, seq, o, lse, ws.ptr, ws.nbytes)
    for n in ([10, 290], [250, 0], [1, 1]):
        seq.copy_(dev(offsets(n)))
        q.copy_(bf16(q.shape, rng))
        o.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        ws.check()
        check_prompt(q, k, v, offsets(n), offsets(n), True, o, lse)


# --------------------------------------------------------------------------------------------- the cache

class Cache:
    """A pool on the host and on the device, sequences in it, and the library's calls on them."""

    def __init__(self, rng, lens, block, H, H_kv, d, new=None, extra=2, width=None, **params):
        self.lens, self.block, self.H, self.H_kv, self.d = [int(x) for x in lens], block, H, H_kv, d
        self.n_blocks = sum(-(-t // block) for t in self.lens) + extra
        self.host = make_pool(rng, self.n_blocks, H_kv, block, d)
        self.table = make_table(rng, self.lens, block, self.n_blocks, width)
        self.w = rng.random((self.n_blocks, H_kv, block)).astype(np.float32)
        self.pool = {n: dev(x) for n, x in self.host.items()}
        self.w_dev = dev(self.w)
        self.seq = offsets(new if new is not None else [0] * len(lens))
        self.p = sda.cache_params(B=len(lens), H=H, H_kv=H_kv, d=d, block=block, n_blocks=self.n_blocks,
                                  max_blocks=self.table.shape[1], rows=int(self.seq[-1]),
                                  max_new=int(np.max(np.diff(self.seq))), **params)
        self.ws = sda.Workspace(self.p)

    def args(self):
        return (dev(np.array(self.lens, np.int32)), dev(self.table), self.pool["k_codes"], self.pool["v_codes"],
                self.pool["k_scale"], self.pool["v_scale"])

    def free_slots_hold_nan(self):
        """NaN codes in every slot that holds no token."""
        used = np.zeros((self.n_blocks, self.block), bool)
        for b, t in enumerate(self.lens):
            for i in range(t):
                used[self.table[b, i // self.block], i % self.block] = True
        for n in ("k_codes", "v_codes"):
            self.host[n][np.nonzero(~used)[0], :, np.nonzero(~used)[1]] = 0x7F
            self.pool[n] = dev(self.host[n])

    def append(self, k, v, w=True):
        sda.sda_cache_append(self.p, k, v, dev(self.seq), *self.args(), self.w_dev if w else None, self.ws.ptr,
                             self.ws.nbytes)

    def attend(self, q, w_in=None, w_out=None, stream=None):
        o = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
        sda.sda_cache_attn_fwd(self.p, q, dev(self.seq), *self.args(), w_in, w_out, o, self.ws.ptr, self.ws.nbytes, stream)
        return o

    def check_pool(self):
        for n in self.host:
            got = self.pool[n].cpu().numpy()
            assert np.array_equal(got, self.host[n]), f"{n}: {np.sum(got != self.host[n])} values differ"


APPENDS = [
    # tokens after the call, new ones, block, H_kv, d
    ([1], [1], 16, 1, 64),
    ([16, 17, 1, 40], [1, 1, 1, 1], 16, 2, 128),
    ([64, 65, 130, 63], [1, 1, 1, 1], 64, 3, 128),
    ([200, 5, 129, 128], [200, 5, 2, 128], 128, 2, 128),
    ([100, 70, 33, 7], [37, 0, 33, 2], 32, 2, 64),        # a sequence without new rows
    ([300, 40], [299, 40], 16, 5, 64),
    ([150, 64], [100, 64], 64, 1, 64),
    ([131], [3], 128, 2, 64),
]


@pytest.mark.parametrize("lens,new,block,H_kv,d", APPENDS)
def test_append(lens, new, block, H_kv, d):
    rng = np.random.default_rng(sum(lens) + block)
    c = Cache(rng, lens, block, H_kv, H_kv, d, new)
    mag = np.exp2(rng.integers(-12, 6, (c.seq[-1], H_kv, 1)))
    k, v = (bf16((c.seq[-1], H_kv, d), rng).float() * torch.from_numpy(mag).float() for _ in range(2))
    if len(k) > 1:
        k[0], v[-1] = 0.0, -0.0                   # zero tokens
    k, v = k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV)
    O.append(f64(k), f64(v), c.seq, c.lens, c.table, block, c.host, c.w)
    c.append(k, v)
    c.ws.check()
    c.check_pool()
    assert np.array_equal(c.w_dev.cpu().numpy(), c.w)
    c.append(k, v)                                # the same rows again: nothing changes
    c.check_pool()


def test_append_extreme_values():
    """Zeros only, the smallest and largest numbers, infinities and NaN, scales of a foreign quantiser."""
    rng = np.random.default_rng(11)
    c = Cache(rng, [20, 20, 20, 20, 20], 16, 1, 1, 64, [20] * 5)
    k = bf16((100, 1, 64), rng)
    k[:20] = 0
    k[20:40] *= 2.0 ** -120
    k[40:60] = (k[40:60].float() * 2.0 ** 125).clamp(-3.3e38, 3.3e38).to(torch.bfloat16)
    k[60, 0, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    k[80:100] = 2.0 ** -133
    k = k.to(DEV)
    O.append(f64(k), f64(k), c.seq, c.lens, c.table, 16, c.host)
    c.append(k, k, w=False)
    c.ws.check()
    c.check_pool()
    # a scale that is no power of two, larger and smaller than the new token's
    d = Cache(rng, [5, 5], 16, 1, 1, 64, [1, 1])
    for b, s in ((0, 0.3), (1, 0.0007)):
        for n in ("k_scale", "v_scale"):
            d.host[n][d.table[b, 0]] = s
            d.pool[n] = dev(d.host[n])
    x = bf16((2, 1, 64), rng).to(DEV)
    O.append(f64(x), f64(x), d.seq, d.lens, d.table, 16, d.host)
    d.append(x, x, w=False)
    d.check_pool()


ATTENDS = [
    # tokens, new rows, block, H, H_kv, d
    ([1], [1], 16, 1, 1, 64),
    ([1, 16, 17, 33], [1, 1, 1, 1], 16, 4, 2, 128),
    ([31, 32, 33, 64, 65], [1, 1, 1, 1, 1], 32, 8, 2, 64),
    ([700, 3, 129], [1, 1, 1], 64, 8, 1, 128),
    ([1000, 40], [4, 3], 16, 10, 2, 128),                # 20 rows of a key head: two row tiles
    ([2, 500, 64], [5, 9, 2], 32, 4, 2, 64),             # more new rows than tokens: the first see nothing
    ([0, 70, 0], [1, 1, 0], 64, 4, 4, 128),              # no token; no row
    ([3000], [1], 128, 16, 1, 128),
    ([5000, 1], [1, 1], 64, 3, 3, 64),
    ([260], [70], 128, 4, 2, 128),                       # many row tiles
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("lens,new,block,H,H_kv,d", ATTENDS)
def test_cache_attention(lens, new, block, H, H_kv, d, weights):
    rng = np.random.default_rng(sum(lens) + block + H)
    c = Cache(rng, lens, block, H, H_kv, d, new, weights=weights)
    c.free_slots_hold_nan()
    q = bf16((c.seq[-1], H, d), rng)
    if len(q) > 1:
        q[0] *= 2.0 ** -60                        # a row of tiny numbers: a uniform average
    q = q.to(DEV)
    w_in = dev(rng.random(c.w.shape).astype(np.float32)) if weights else None
    w_out = torch.full(c.w.shape, 7.0, device=DEV) if weights else None
    o = c.attend(q, w_in, w_out)
    c.ws.check()
    want, spread, w = O.cache_attention(f64(q), c.seq, c.lens, c.table, block, c.host)
    size = max([score_size(f64(q), O.cache_values(c.host, "k", c.table[b], t, block, h))
                for b, t in enumerate(c.lens) if t for h in range(H_kv)] or [0.0])
    tol = attention_tolerance(want, spread, size, d, U_F16)
    err = np.abs(f64(o) - want)
    assert np.all(err <= tol), f"o: {np.max(err - tol):.3e} over the bound, worst error {err.max():.3e}"
    assert torch.equal(o, c.attend(q, w_in, w_out))       # and the same bits again
    if weights:
        expect = np.full(c.w.shape, 7.0)
        bound = np.zeros(c.w.shape)
        p_error = 2 * (2 * (d + 8) * U_F32 * size + 2.0 ** -20)
        for b, t in enumerate(c.lens):
            i = np.arange(t)
            blk = c.table[b, i // block]
            for h in range(H_kv):
                expect[blk, h, i % block] = f64(w_in)[blk, h, i % block] + w[b][h]
                bound[blk, h, i % block] = w[b][h] * (p_error + new[b] * (H // H_kv) * U_F32) + 2 * U_F32 * expect[blk, h, i % block]
        err = np.abs(f64(w_out) - expect)
        assert np.all(err <= bound), f"w: worst error {err.max():.3e}"
        o2 = c.attend(q, w_out, w_out)                    # in place, on top of the first call's
        assert torch.equal(o, o2)
        twice = np.where(expect == 7, 7, expect)
        for b, t in enumerate(c.lens):
            i = np.arange(t)
            blk = c.table[b, i // block]
            for h in range(H_kv):
                twice[blk, h, i % block] += w[b][h]
        assert np.all(np.abs(f64(w_out) - twice) <= 2 * bound + 2 * U_F32 * twice)


def test_cache_attention_weights_from_nothing():
    rng = np.random.default_rng(12)
    c = Cache(rng, [100, 50], 32, 4, 2, 64, [2, 1], weights=True)
    q = bf16((3, 4, 64), rng).to(DEV)
    w_out = torch.full(c.w.shape, float("nan"), device=DEV)
    c.attend(q, None, w_out)
    total = sum(w_out[c.table[b, :-(-t // 32)]].double().nan_to_num().sum().item() for b, t in enumerate(c.lens))
    assert abs(total - 3 * 4) < 1e-4              # probabilities of 3 rows and 4 heads: 12 in all, 150 tokens' fp32 sums
    assert torch.isnan(w_out[c.table[0, 3], :, 4:]).all()  # free slots of the last block


def test_cache_attention_unequal_scales():
    """V's scales over 60 binades, the largest block with no weight: fp16 has to hold the rest all the same."""
    rng = np.random.default_rng(13)
    d, block = 64, 16
    c = Cache(rng, [200], block, 2, 1, d, [1])
    c.host["v_scale"][:] = np.exp2(rng.integers(-30, 31, c.host["v_scale"].shape)).astype(np.float32)
    big = c.table[0, 3]
    c.host["v_scale"][big] = 2.0 ** 100
    c.host["k_codes"][big] = 0xFE                 # -448: no weight under a query of ones
    zero = c.table[0, 5]
    c.host["v_codes"][zero], c.host["v_scale"][zero] = 0, 2.0 ** -126
    c.pool = {n: dev(x) for n, x in c.host.items()}
    q = torch.ones(1, 2, d, dtype=torch.bfloat16, device=DEV) * 4
    o = c.attend(q)
    want, spread, _ = O.cache_attention(f64(q), c.seq, c.lens, c.table, block, c.host)
    size = score_size(f64(q), np.concatenate([O.cache_values(c.host, "k", c.table[0], 200, block, 0)]))
    assert np.all(np.abs(f64(o) - want) <= attention_tolerance(want, spread, size, d, U_F16))


def test_cache_bad_device_arguments_are_reported_and_stay_in_range():
    rng = np.random.default_rng(14)
    for bad in ("table_low", "table_high", "lens_high", "lens_low", "seq_high", "seq_down", "new"):
        c = Cache(rng, [40, 50], 16, 2, 1, 64, [1, 1], weights=True, keep=16, recent=2)
        lens, table, seq = np.array(c.lens, np.int32), c.table.copy(), c.seq.copy()
        if bad == "table_low":
            table[1, 1:] = -5
        elif bad == "table_high":
            table[0], table[1, 3] = c.n_blocks, (1 << 31) - 1
        elif bad == "lens_high":
            lens[1] = (1 << 31) - 1
        elif bad == "lens_low":
            lens[0] = -(1 << 31)
        elif bad == "seq_high":
            seq[2] = 1 << 30
        elif bad == "seq_down":
            seq[1], seq[2] = 2, 1
        else:
            seq = np.array([0, 2, 2], np.int32)   # two rows where max_new is 1
        if bad == "lens_high":                    # blocks that the table names have to be in the pool
            table[1] = c.table[1, 0]
        args = (dev(lens), dev(table), *c.args()[2:])
        x, q = bf16((2, 1, 64), rng).to(DEV), bf16((2, 2, 64), rng).to(DEV)
        calls = [lambda: sda.sda_cache_append(c.p, x, x, dev(seq), *args, c.w_dev, c.ws.ptr, c.ws.nbytes),
                 lambda: sda.sda_cache_attn_fwd(c.p, q, dev(seq), *args, None, c.w_dev, torch.empty_like(q), c.ws.ptr,
                                                c.ws.nbytes)]
        if not bad.startswith("seq") and bad != "new":
            dst = dev(np.array([[0], [1]], np.int32))
            kept, n = torch.empty((2, 1, 16), dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
            calls.append(lambda: sda.sda_cache_evict(c.p, *args, c.w_dev, dst, kept, n, c.ws.ptr, c.ws.nbytes))
        for i, call in enumerate(calls):
            call()
            with pytest.raises(sda.SdaError) as e:
                c.ws.check()
            assert e.value.code == -3, (bad, i)
            c.ws.check()


EVICTS = [
    # tokens, block, H_kv, d, keep, recent
    ([1], 16, 1, 64, 1, 0),
    ([40, 16, 1, 17], 16, 2, 128, 16, 4),
    ([100, 300, 0, 64], 32, 2, 64, 50, 50),               # only the newest; an empty sequence
    ([1000, 129], 64, 3, 128, 200, 0),
    ([700], 128, 1, 128, 300, 33),
    ([2500, 2499], 64, 2, 64, 2498, 10),
]


@pytest.mark.parametrize("weights", ["random", "ties", "equal", "special"])
@pytest.mark.parametrize("lens,block,H_kv,d,keep,recent", EVICTS)
def test_evict(lens, block, H_kv, d, keep, recent, weights):
    rng = np.random.default_rng(sum(lens) + block)
    width = -(-keep // block)
    c = Cache(rng, lens, block, H_kv, H_kv, d, extra=len(lens) * width + 1, keep=keep, recent=recent)
    shape = c.w.shape
    c.w = {"random": rng.normal(size=shape), "ties": rng.integers(0, 4, shape) / 4, "equal": np.zeros(shape),
           "special": rng.choice([0.0, -0.0, np.inf, -np.inf, np.nan, 1e-40, 3.0], shape)}[weights].astype(np.float32)
    c.w_dev = dev(c.w)
    free = [b for b in rng.permutation(c.n_blocks) if b not in c.table]
    dst = np.full((len(lens), width), -1, np.int32)
    for b, t in enumerate(lens):
        n = -(-min(t, keep) // block)
        dst[b, :n], free = free[:n], free[n:]
    c.free_slots_hold_nan()
    kept, n = O.evict(c.lens, c.table, block, c.host, c.w, dst, keep, recent)
    got_kept = torch.full((len(lens), H_kv, keep), 7, dtype=torch.int32, device=DEV)
    got_n = torch.full((len(lens),), 7, dtype=torch.int32, device=DEV)
    sda.sda_cache_evict(c.p, *c.args(), c.w_dev, dev(dst), got_kept, got_n, c.ws.ptr, c.ws.nbytes)
    c.ws.check()
    assert np.array_equal(got_n.cpu().numpy(), n)
    assert np.array_equal(got_kept.cpu().numpy(), kept)
    c.check_pool()
    assert np.array_equal(c.w_dev.cpu().numpy(), c.w, equal_nan=True)


def test_evict_longer_than_shared_memory_holds():
    """70,000 tokens: more keys than the selection keeps in shared memory. Positions against a stable sort."""
    rng = np.random.default_rng(15)
    c = Cache(rng, [70000, 49153], 128, 1, 1, 64, extra=200, keep=10000, recent=100)
    c.w = (rng.integers(0, 500, c.w.shape) / 8).astype(np.float32)
    c.w_dev = dev(c.w)
    free = [b for b in range(c.n_blocks) if b not in c.table]
    dst = np.array([free[:79], free[79:158]], np.int32)
    kept, n = torch.empty((2, 1, 10000), dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    sda.sda_cache_evict(c.p, *c.args(), c.w_dev, dev(dst), kept, n, c.ws.ptr, c.ws.nbytes)
    c.ws.check()
    for b, t in enumerate(c.lens):
        i = np.arange(t)
        w = c.w[c.table[b, i // 128], 0, i % 128]
        older = np.argsort(-w[:t - 100], kind="stable")[:9900]
        assert np.array_equal(kept[b, 0].cpu().numpy(), np.concatenate([np.sort(older), i[t - 100:]]))


def test_pool_of_more_than_4_gib():
    """Blocks behind the 32-bit byte offsets of the codes."""
    n_blocks, H_kv, block, d = 300_000, 1, 128, 128
    rng = np.random.default_rng(16)
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB of device memory")
    pool = {n: torch.zeros((n_blocks, H_kv, block, d), dtype=torch.uint8, device=DEV) for n in ("k_codes", "v_codes")}
    pool |= {n: torch.ones((n_blocks, H_kv), device=DEV) for n in ("k_scale", "v_scale")}
    w = torch.zeros((n_blocks, H_kv, block), device=DEV)
    table = np.array([[n_blocks - 1, n_blocks - 3]], np.int32)
    lens = [200]
    p = sda.cache_params(B=1, H=4, H_kv=1, d=d, block=block, n_blocks=n_blocks, max_blocks=2, rows=200, max_new=200,
                         weights=True, keep=100, recent=10)
    ws = sda.Workspace(p)
    k, v, q = (bf16((200, h, d), rng).to(DEV) for h in (1, 1, 4))
    seq, args = dev(offsets([200])), (dev(np.array(lens, np.int32)), dev(table), *pool.values())
    sda.sda_cache_append(p, k, v, seq, *args, w, ws.ptr, ws.nbytes)
    o = torch.empty_like(q)
    sda.sda_cache_attn_fwd(p, q, seq, *args, None, w, o, ws.ptr, ws.nbytes)
    dst = np.array([[n_blocks - 2]], np.int32)
    kept, n = torch.empty((1, 1, 100), dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    w_before = w[[n_blocks - 1, n_blocks - 3]].cpu().numpy()
    sda.sda_cache_evict(p, *args, w, dev(dst), kept, n, ws.ptr, ws.nbytes)
    ws.check()
    host = {m: x[-3:].cpu().numpy() for m, x in pool.items()}     # the last three blocks: 2, 0 (of 3) hold the tokens
    small = np.array([[2, 0]], np.int32)
    want = {m: np.zeros_like(x) for m, x in host.items()}
    O.append(f64(k), f64(v), [0, 200], lens, small, block, want)
    for m in ("k_codes", "v_codes", "k_scale", "v_scale"):
        assert np.array_equal(host[m][[2, 0]][:, :, :72] if "codes" in m else host[m][[2, 0]],
                              want[m][[2, 0]][:, :, :72] if "codes" in m else want[m][[2, 0]])
    ref, spread, _ = O.cache_attention(f64(q), [0, 200], lens, small, block, want)
    size = score_size(f64(q), O.cache_values(want, "k", small[0], 200, block, 0))
    assert np.all(np.abs(f64(o) - ref) <= attention_tolerance(ref, spread, size, d, U_F16))
    flat = w_before[:, 0].reshape(-1)[:200]
    assert np.array_equal(kept[0, 0].cpu().numpy(), O.kept_positions(flat, 200, 100, 10))


def test_cache_two_graphs_with_their_own_workspaces():
    """Two captured steps of two caches replay side by side on two streams."""
    rng = np.random.default_rng(17)
    steps = []
    for lens in ([900, 33], [64, 2000]):
        c = Cache(rng, lens, 32, 8, 2, 64, [1, 1], weights=True)
        q = bf16((2, 8, 64), rng).to(DEV)
        o, w_out = torch.empty_like(q), torch.zeros(c.w.shape, device=DEV)
        a = (q, dev(c.seq), *c.args(), None, w_out, o)
        sda.sda_cache_attn_fwd(c.p, *a, c.ws.ptr, c.ws.nbytes)
        torch.cuda.synchronize()
        first = o.clone(), w_out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sda.sda_cache_attn_fwd(c.p, *a, c.ws.ptr, c.ws.nbytes)
        o.zero_(), w_out.zero_()
        steps.append((c, a, g, first, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, a, g, first, s in steps:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, a, g, first, s in steps:
        c.ws.check()
        assert torch.equal(a[-1], first[0]) and torch.equal(a[-2], first[1])


def test_serving_run_together():
    """Prompts through the prompt attention into the cache, decoding steps that collect weights, an eviction, and
    more steps on what stayed, each against the oracle on the library's own cache contents."""
    rng = np.random.default_rng(18)
    B, H, H_kv, d, block, steps, keep, recent = 3, 8, 2, 128, 32, 4, 60, 10
    n = [100, 7, 61]
    width, n_blocks = 5, 40
    free = list(rng.permutation(n_blocks))
    table = np.array([[free.pop() for _ in range(width)] for _ in range(B)], np.int32)
    dst = np.array([[free.pop() for _ in range(-(-keep // block))] for _ in range(B)], np.int32)
    made = make_pool(rng, n_blocks, H_kv, block, d)
    pool = {m: dev(made[m]) for m in ("k_codes", "v_codes", "k_scale", "v_scale")}   # in the calls' order
    w = torch.full((n_blocks, H_kv, block), float("nan"), device=DEV)

    def params(rows, max_new, table):
        return sda.cache_params(B=B, H=H, H_kv=H_kv, d=d, block=block, n_blocks=n_blocks, max_blocks=table.shape[1],
                                rows=rows, max_new=max_new, weights=True, keep=keep, recent=recent)

    def host():
        return {m: x.cpu().numpy() for m, x in pool.items()}

    seq = offsets(n)
    q, k, v = (bf16((seq[-1], h, d), rng).to(DEV) for h in (H, H_kv, H_kv))
    o, lse = run_prompt(q, k, v, seq, seq, True)
    check_prompt(q, k, v, seq, seq, True, o, lse)
    p = params(int(seq[-1]), max(n), table)
    ws = sda.Workspace(p)
    sda.sda_cache_append(p, k, v, dev(seq), dev(np.array(n, np.int32)), dev(table), *pool.values(), w, ws.ptr, ws.nbytes)
    ws.check()
    for b in range(B):                            # the cache holds the prompt within its rounding
        for h in range(H_kv):
            got = O.cache_values(host(), "k", table[b], n[b], block, h)
            x = f64(k)[seq[b]:seq[b + 1], h]
            assert np.all(np.abs(got - x) <= np.maximum(np.abs(x) / 16, host()["k_scale"].max() * 2.0 ** -10))

    def decode(table, lens, ws, p):
        seq1 = offsets([1] * B)
        q, k, v = (bf16((B, h, d), rng).to(DEV) for h in (H, H_kv, H_kv))
        args = (dev(np.array(lens, np.int32)), dev(table), *pool.values())
        o = torch.empty_like(q)
        sda.sda_cache_append(p, k, v, dev(seq1), *args, w, ws.ptr, ws.nbytes)
        sda.sda_cache_attn_fwd(p, q, dev(seq1), *args, w, w, o, ws.ptr, ws.nbytes)
        ws.check()
        want, spread, wt = O.cache_attention(f64(q), seq1, lens, table, block, host())
        size = max(score_size(f64(q), O.cache_values(host(), "k", table[b], lens[b], block, h))
                   for b in range(B) for h in range(H_kv))
        assert np.all(np.abs(f64(o) - want) <= attention_tolerance(want, spread, size, d, U_F16))
        return wt

    lens = list(n)
    p1 = params(B, 1, table)
    ws1 = sda.Workspace(p1)
    collected = [np.zeros((H_kv, t)) for t in lens]
    for _ in range(steps):
        lens = [t + 1 for t in lens]
        wt = decode(table, lens, ws1, p1)
        collected = [np.pad(c, ((0, 0), (0, 1))) + x for c, x in zip(collected, wt)]
    got_w = w.cpu().numpy()
    for b, t in enumerate(lens):
        i = np.arange(t)
        assert np.allclose(got_w[table[b, i // block], :, i % block].T, collected[b], rtol=1e-4, atol=1e-7)
    pool_before, w_before = host(), got_w.copy()
    kept, n_dst = torch.empty((B, H_kv, keep), dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
    sda.sda_cache_evict(p1, dev(np.array(lens, np.int32)), dev(table), *pool.values(), w, dev(dst), kept, n_dst, ws1.ptr,
                        ws1.nbytes)
    ws1.check()
    want_kept, want_n = O.evict(lens, table, block, pool_before, w_before, dst, keep, recent)
    assert np.array_equal(kept.cpu().numpy(), want_kept) and np.array_equal(n_dst.cpu().numpy(), want_n)
    for m, x in host().items():
        assert np.array_equal(x, pool_before[m]), m
    # further steps on the target blocks, with room for them in a wider table
    more = np.concatenate([dst, [[free.pop()] for _ in range(B)]], 1).astype(np.int32)
    p2 = params(B, 1, more)
    ws2 = sda.Workspace(p2)
    lens = [int(x) for x in want_n]
    for _ in range(6):
        lens = [t + 1 for t in lens]
        decode(more, lens, ws2, p2)


@pytest.mark.parametrize("call", ["prompt", "cache"])
def test_wait_that_runs_out_is_reported_and_the_next_call_works(call):
    """With a limit of 0 a wait gives up unless its phase is already complete: the kernel reports it, drains and
    ends; afterwards the same call works on the same workspace. (The cache kernel's loads may all have landed before
    its waits: then nothing runs out, and the output is right.)"""
    rng = np.random.default_rng(19)
    if call == "prompt":
        q, k, v = (bf16((700, h, 128), rng).to(DEV) for h in (4, 2, 2))
        p = sda.prompt_params(n_seq=2, rows_q=700, rows_k=700, H=4, H_kv=2, d=128)
        ws, seq, o = sda.Workspace(p), dev(offsets([500, 200])), torch.empty_like(q)
        run = lambda: sda.sda_prompt_attn_fwd(p, q, k, v, seq, seq, o, None, ws.ptr, ws.nbytes)  # noqa: E731
    else:
        c = Cache(rng, [3000, 40], 64, 8, 2, 128, [1, 1])
        q = bf16((2, 8, 128), rng).to(DEV)
        ws, o = c.ws, torch.empty_like(q)
        a = (q, dev(c.seq), *c.args(), None, None, o)
        run = lambda: sda.sda_cache_attn_fwd(c.p, *a, ws.ptr, ws.nbytes)  # noqa: E731
    run()
    ws.check()
    want = o.clone()
    before = sda.sda_set_attention_wait_limit_ns(0)
    try:
        run()
        try:
            ws.check()
            assert call == "cache" and torch.equal(o, want)
        except sda.SdaError as e:
            assert e.code == -7
    finally:
        sda.sda_set_attention_wait_limit_ns(before)
    ws.check()
    o.zero_()
    run()
    ws.check()
    assert torch.equal(o, want)


def test_cache_shared_prefix_and_many_short_sequences():
    """Blocks shared by sequences (a common prefix), more sequences than a warp has lanes, some without rows, some
    without tokens; block tables wide enough that the work is split."""
    rng = np.random.default_rng(20)
    B, H, H_kv, d, block = 70, 4, 2, 64, 16
    lens = [int(x) for x in rng.integers(0, 90, B)]
    lens[3], lens[40] = 700, 0
    new = [int(x) for x in rng.integers(0, 3, B)]
    c = Cache(rng, lens, block, H, H_kv, d, new, width=64)
    for b in range(5, 60, 7):                     # the first block of some is that of sequence 3
        if lens[b]:
            c.table[b, 0] = c.table[3, 0]
    q = bf16((int(c.seq[-1]), H, d), rng).to(DEV)
    o = c.attend(q)
    c.ws.check()
    want, spread, _ = O.cache_attention(f64(q), c.seq, c.lens, c.table, block, c.host)
    size = max(score_size(f64(q), O.cache_values(c.host, "k", c.table[b], t, block, h))
               for b, t in enumerate(c.lens) if t for h in range(H_kv))
    assert np.all(np.abs(f64(o) - want) <= attention_tolerance(want, spread, size, d, U_F16))


def test_serving_rows_apart():
    """q, k, v of the cache calls as slices of one projection's rows, o as a slice of a wider tensor."""
    rng = np.random.default_rng(21)
    H, H_kv, d, block, lens, new = 4, 2, 64, 16, [50, 33], [2, 1]
    n = sum(new)
    rows = bf16((n, (H + 2 * H_kv) * d), rng).to(DEV)
    q, k, v = (x.unflatten(1, (h, d)) for x, h in zip(rows.split([H * d, H_kv * d, H_kv * d], 1), (H, H_kv, H_kv)))
    wide = torch.full((n, 2 * H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    ld = rows.shape[1]
    c = Cache(rng, lens, block, H, H_kv, d, new, ld_q=ld, ld_k=ld, ld_v=ld, ld_o=2 * H * d)
    O.append(f64(k), f64(v), c.seq, c.lens, c.table, block, c.host)
    c.append(k, v, w=False)
    c.check_pool()
    o = wide[:, H:]
    sda.sda_cache_attn_fwd(c.p, q, dev(c.seq), *c.args(), None, None, o, c.ws.ptr, c.ws.nbytes)
    c.ws.check()
    assert torch.all(wide[:, :H] == 7)
    want, spread, _ = O.cache_attention(f64(q), c.seq, c.lens, c.table, block, c.host)
    size = max(score_size(f64(q), O.cache_values(c.host, "k", c.table[b], t, block, h))
               for b, t in enumerate(lens) for h in range(H_kv))
    assert np.all(np.abs(f64(o) - want) <= attention_tolerance(want, spread, size, d, U_F16))


@pytest.mark.parametrize("n", [[1], [100], [513], [64, 65], [3] * 40])
def test_prompt_every_row_is_written_every_time(n):
    """The search for a CTA's next tile says "none" and then "this one" in the same place; if the first store could
    land last, a tile's rows would stay unwritten without a report. Many calls, each into fresh marks."""
    rng = np.random.default_rng(30)
    sq = offsets(n)
    q, k, v = (bf16((int(sq[-1]), h, 64), rng).to(DEV) for h in (8, 2, 2))
    p = sda.prompt_params(n_seq=len(n), rows_q=len(q), rows_k=len(q), H=8, H_kv=2, d=64)
    ws, seq = sda.Workspace(p), dev(sq)
    first, _ = run_prompt(q, k, v, sq, sq, True)
    assert not torch.any(torch.isnan(first))
    o = [torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(200)]
    for x in o:
        sda.sda_prompt_attn_fwd(p, q, k, v, seq, seq, x, None, ws.ptr, ws.nbytes)
    ws.check()
    assert all(torch.equal(x, first) for x in o)


WIDE_RANGES = [
    # tokens, new rows, block, H, H_kv, d
    ([300, 40], [1, 1], 32, 4, 2, 64),            # a CTA per unit
    ([4097], [1], 64, 4, 1, 128),                 # split over many CTAs, a CTA joins a row
    ([900, 30] * 12, [1] * 24, 64, 4, 2, 64),     # split, a warp joins a row
    ([3000, 70], [2, 1], 16, 16, 1, 128),         # 16 rows to a tile, blocks of half a tile
]


def check_cache_attention(c, q):
    o = c.attend(q)
    c.ws.check()
    want, spread, _ = O.cache_attention(f64(q), c.seq, c.lens, c.table, c.block, c.host)
    size = max(score_size(f64(q), O.cache_values(c.host, "k", c.table[b], t, c.block, h))
               for b, t in enumerate(c.lens) if t for h in range(c.H_kv))
    tol = attention_tolerance(want, spread, size, c.d, U_F16)
    err = np.abs(f64(o) - want)
    assert np.all(err <= tol), f"worst error {np.max(err / tol):.2f} of the bound"
    assert torch.equal(o, c.attend(q))


@pytest.mark.parametrize("gap", [14, 16, 18, 20, 30, 45])
@pytest.mark.parametrize("lens,new,block,H,H_kv,d", WIDE_RANGES)
def test_cache_attention_dominant_token_that_holds_nothing(lens, new, block, H, H_kv, d, gap):
    """Token 0 `gap` nats above the rest with a V of zero: the output is that of all the others, whose weights are
    far below fp16's range under the row's largest. The bound counts a rounding of 2^-11 for each of them."""
    rng = np.random.default_rng(gap)
    c = Cache(rng, lens, block, H, H_kv, d, new)
    c.host["k_scale"][:] = 2.0 ** -7
    top = 2.0 if gap > 28 else 1.0                # q: the same number everywhere, so that a constant K gives its score
    for b in range(len(lens)):
        c.host["k_codes"][c.table[b, 0], :, 0] = O.encode_e4m3(np.float32(gap * 2.0 ** 7 / (top * d ** 0.5)))
        c.host["v_codes"][c.table[b, 0], :, 0] = 0
    c.pool = {n: dev(x) for n, x in c.host.items()}
    c.free_slots_hold_nan()
    check_cache_attention(c, torch.full((int(c.seq[-1]), H, d), top, dtype=torch.bfloat16, device=DEV))


@pytest.mark.parametrize("binades", [20, 40, 60])
@pytest.mark.parametrize("lens,new,block,H,H_kv,d", WIDE_RANGES)
def test_cache_attention_block_scaled_for_another_channel(lens, new, block, H, H_kv, d, binades):
    """A block whose V is scaled far above the others' for one channel and zero elsewhere: the other channels' output
    comes from the other blocks alone."""
    rng = np.random.default_rng(binades)
    c = Cache(rng, lens, block, H, H_kv, d, new)
    for b in range(len(lens)):
        blk = c.table[b, (lens[b] - 1) // block // 2]
        c.host["v_scale"][blk] = 2.0 ** (binades - 7)
        c.host["v_codes"][blk] = 0
        c.host["v_codes"][blk, :, ::3, 5] = 0x7E  # 448 in one channel of every third token
    c.pool = {n: dev(x) for n, x in c.host.items()}
    c.free_slots_hold_nan()
    check_cache_attention(c, bf16((int(c.seq[-1]), H, d), rng).to(DEV))


@pytest.mark.parametrize("code", [176.0, 192.0])
@pytest.mark.parametrize("lens,new,block,H,H_kv,d", WIDE_RANGES)
def test_cache_attention_scale_makes_up_for_a_tiny_weight(lens, new, block, H, H_kv, d, code):
    """A block whose probabilities are below 2^-126 of the row's largest, with V's scale as far above the others':
    it takes its share of the output."""
    rng = np.random.default_rng(int(code))
    c = Cache(rng, lens, block, H, H_kv, d, new)
    c.host["k_scale"][:] = 2.0 ** -7
    c.host["v_scale"][:] = 2.0 ** -20
    for b in range(len(lens)):
        blk = c.table[b, (lens[b] - 1) // block // 2]
        c.host["k_codes"][blk], c.host["k_scale"][blk] = O.encode_e4m3(np.float32(-code)), 2.0 ** -5
        nats = 2 * code * 2.0 ** -5 * d ** 0.5    # under q = 2 everywhere
        while nats > 96:                          # keep the scale within fp32: d = 128
            c.host["k_scale"][blk] /= 2
            nats /= 2
        if nats < 80:
            c.host["k_codes"][blk] = O.encode_e4m3(np.float32(-code * 88 / nats))
            nats = 88
        c.host["v_scale"][blk] = 2.0 ** (round(nats / np.log(2)) - 20)
    c.pool = {n: dev(x) for n, x in c.host.items()}
    c.free_slots_hold_nan()
    check_cache_attention(c, torch.full((int(c.seq[-1]), H, d), 2.0, dtype=torch.bfloat16, device=DEV))


def test_cache_codes_in_torchs_own_type():
    """torch.float8_e4m3fn codes are the same bytes."""
    rng = np.random.default_rng(31)
    c = Cache(rng, [50, 33], 16, 4, 2, 64, [2, 1])
    q, k, v = (bf16((3, h, 64), rng).to(DEV) for h in (4, 2, 2))
    O.append(f64(k), f64(v), c.seq, c.lens, c.table, 16, c.host)
    for n in ("k_codes", "v_codes"):
        c.pool[n] = c.pool[n].view(torch.float8_e4m3fn)
    c.append(k, v, w=False)
    o = c.attend(q)
    for n in ("k_codes", "v_codes"):
        c.pool[n] = c.pool[n].view(torch.uint8)
    c.check_pool()
    assert torch.equal(o, c.attend(q))


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("value", [-1.0, float("nan"), float("inf"), 0.0])
def test_cache_scales_outside_their_range_are_reported(which, value):
    """Negative, NaN and infinite scales of a sequence's blocks; zero is a scale, and blocks of nobody do not count."""
    rng = np.random.default_rng(32)
    for at, seen in ((0, True), (1, True), (None, False)):       # the first block, the last one, one of nobody
        c = Cache(rng, [60, 40], 32, 2, 1, 64, [1, 1], keep=32, recent=2, extra=4)
        free = [b for b in range(c.n_blocks) if b not in c.table]
        blk = free.pop() if at is None else c.table[0, at]
        c.host[which][blk] = value
        c.pool[which] = dev(c.host[which])
        q, x = bf16((2, 2, 64), rng).to(DEV), bf16((2, 1, 64), rng).to(DEV)
        dst = np.array([[free.pop()], [free.pop()]], np.int32)
        kept, n = torch.empty((2, 1, 32), dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
        c.w[:] = 0
        c.w[c.table[0, 0]] = 1                                   # tokens of the first block stay, and the newest two
        c.w_dev = dev(c.w)
        calls = [lambda: c.attend(q),
                 lambda: sda.sda_cache_evict(c.p, *c.args(), c.w_dev, dev(dst), kept, n, c.ws.ptr, c.ws.nbytes),
                 lambda: c.append(x, x, w=False)]
        for i, call in enumerate(calls):
            call()
            # an append touches the last block alone
            if value == 0.0 or not seen or (i == 2 and at == 0):
                c.ws.check()
                continue
            with pytest.raises(sda.SdaError) as e:
                c.ws.check()
            assert e.value.code == -3, (i, at)
            c.ws.check()


def test_cache_scale_of_zero():
    """A block whose scale is zero holds zeros: under attention, under an append that goes on in it, and under
    eviction beside others."""
    rng = np.random.default_rng(33)
    c = Cache(rng, [60, 40], 32, 2, 1, 64, [1, 1], keep=32, recent=16, extra=4)
    for n in ("k_scale", "v_scale"):
        c.host[n][c.table[0, 1]] = 0.0
    c.host["v_scale"][c.table[1, :2]] = 0.0                       # all of a sequence's V
    c.pool = {n: dev(x) for n, x in c.host.items()}
    q, k, v = (bf16((2, h, 64), rng).to(DEV) for h in (2, 1, 1))
    check_cache_attention(c, q)
    assert torch.all(c.attend(q)[1] == 0)
    free = [b for b in range(c.n_blocks) if b not in c.table]
    dst = np.array([[free[0]], [-1]], np.int32)                   # one sequence: a block of zeros only has no largest scale
    lens, c.lens = c.lens, [60, 0]
    kept, n = torch.empty((2, 1, 32), dtype=torch.int32, device=DEV), torch.empty(2, dtype=torch.int32, device=DEV)
    want_kept, want_n = O.evict(c.lens, c.table, 32, c.host, c.w, dst, 32, 16)
    sda.sda_cache_evict(c.p, *c.args(), c.w_dev, dev(dst), kept, n, c.ws.ptr, c.ws.nbytes)
    c.ws.check()
    assert np.array_equal(kept.cpu().numpy(), want_kept) and np.array_equal(n.cpu().numpy(), want_n)
    c.check_pool()
    c.lens = lens
    O.append(f64(k), f64(v), c.seq, c.lens, c.table, 32, c.host)
    c.append(k, v, w=False)
    c.ws.check()
    c.check_pool()


def test_eviction_in_a_pool_of_more_than_4_gib():
    """Sources and target behind the 32-bit byte offsets of the codes: codes, scales and weights of the target."""
    n_blocks, H_kv, block, d = 300_000, 1, 128, 128
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB of device memory")
    rng = np.random.default_rng(34)
    host = make_pool(rng, 4, H_kv, block, d)      # the last four blocks; 3 and 1 hold the tokens, 2 is the target
    w = rng.random((4, H_kv, block)).astype(np.float32)
    pool = {n: torch.zeros((n_blocks, *x.shape[1:]), dtype=torch.from_numpy(x).dtype, device=DEV) for n, x in host.items()}
    w_dev = torch.zeros((n_blocks, H_kv, block), device=DEV)
    for n, x in host.items():
        pool[n][-4:] = dev(x)
    w_dev[-4:] = dev(w)
    low = {n: x[:4].clone() for n, x in pool.items()}
    p = sda.cache_params(B=1, H=1, H_kv=H_kv, d=d, block=block, n_blocks=n_blocks, max_blocks=2, keep=100, recent=10)
    ws = sda.Workspace(p)
    table, dst, lens = np.array([[3, 1]], np.int32), np.array([[2]], np.int32), [200]
    kept, n = torch.empty((1, 1, 100), dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    sda.sda_cache_evict(p, dev(np.array(lens, np.int32)), dev(table + n_blocks - 4), pool["k_codes"], pool["v_codes"],
                        pool["k_scale"], pool["v_scale"], w_dev, dev(dst + n_blocks - 4), kept, n, ws.ptr, ws.nbytes)
    ws.check()
    want_kept, want_n = O.evict(lens, table, block, host, w, dst, 100, 10)
    assert np.array_equal(kept.cpu().numpy(), want_kept) and np.array_equal(n.cpu().numpy(), want_n)
    for m, x in pool.items():
        assert np.array_equal(x[-4:].cpu().numpy(), host[m]), m
        assert torch.equal(x[:4], low[m]), m      # where a 32-bit offset would have landed
    assert np.array_equal(w_dev[-4:].cpu().numpy(), w)


@pytest.mark.parametrize("lens,weights", [([500] * 100, False), ([20000, 40], False), ([20000, 40, 7000], True)])
def test_cache_wait_that_runs_out(lens, weights):
    """With a limit of 0 some wait of many calls finds its load not landed: it is reported, every load of the CTA is
    waited for, and the next call on the same workspace is right."""
    rng = np.random.default_rng(35)
    c = Cache(rng, lens, 32, 8, 2, 128, [1] * len(lens), weights=weights)
    q = bf16((len(lens), 8, 128), rng).to(DEV)
    w_out = torch.zeros(c.w.shape, device=DEV) if weights else None
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)      # the cache leaves L2: its loads take their time
    want = c.attend(q, None, w_out)
    c.ws.check()
    want_w = w_out.clone() if weights else None
    before = sda.sda_set_attention_wait_limit_ns(0)
    ran_out = 0
    try:
        for _ in range(50):
            flush.zero_()
            c.attend(q, None, w_out)
            try:
                c.ws.check()
            except sda.SdaError as e:
                assert e.code == -7
                ran_out += 1
                if ran_out == 3:
                    break
    finally:
        sda.sda_set_attention_wait_limit_ns(before)
    assert ran_out, "no wait ran out in 50 calls"
    assert torch.equal(c.attend(q, None, w_out), want)
    c.ws.check()
    assert not weights or torch.equal(w_out, want_w)


@pytest.mark.parametrize("n_seq,H,H_kv,causal", [(1500, 2, 1, True), (1500, 1, 1, False), (20000, 2, 2, True)])
def test_prompt_thousands_of_sequences(n_seq, H, H_kv, causal):
    """Mostly a few tokens each, some empty, some of several tiles, so that a CTA goes through many step counts and
    groups of sequences."""
    rng = np.random.default_rng(36)
    n = rng.integers(0, 7, n_seq)
    n[rng.integers(0, n_seq, 8)] = [600, 300, 290, 257, 256, 129, 128, 127]
    nk = n if causal else rng.integers(0, 7, n_seq)
    sq, sk = offsets(n), offsets(nk)
    q, k, v = (bf16((int(a[-1]), h, 64), rng).to(DEV) for a, h in ((sq, H), (sk, H_kv), (sk, H_kv)))
    o, lse = run_prompt(q, k, v, sq, sk, causal)
    check_prompt(q, k, v, sq, sk, causal, o, lse)


def test_prompt_time_is_linear_in_the_number_of_sequences():
    """16 times as many prompts of 100 tokens take about 16 times as long, the search for a CTA's tiles with them."""
    def time(n):
        q, k, v = (torch.randn(n * 100, h, 64, device=DEV).to(torch.bfloat16) for h in (32, 8, 8))
        p = sda.prompt_params(n_seq=n, rows_q=n * 100, rows_k=n * 100, H=32, H_kv=8, d=64)
        ws, seq, o = sda.Workspace(p), torch.arange(n + 1, dtype=torch.int32, device=DEV) * 100, torch.empty_like(q)
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            sda.sda_prompt_attn_fwd(p, q, k, v, seq, seq, o, None, ws.ptr, ws.nbytes)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        ws.check()
        return best
    few, many = time(256), time(4096)
    assert many < 3 * 16 * few, (few, many)       # 130 times when each tile's search read all offsets anew


@pytest.mark.parametrize("which", [0, 1])
def test_prompt_overlapping_sequences_are_no_work(which):
    """Offsets that go up and down would make every second sequence all the rows: the work stays that of the tensors,
    here none, and the offsets are reported."""
    rng = np.random.default_rng(37)
    T, n_seq = 5000, 40
    q, k, v = (bf16((T, h, 64), rng).to(DEV) for h in (2, 1, 1))
    p = sda.prompt_params(n_seq=n_seq, rows_q=T, rows_k=T, H=2, H_kv=1, d=64)
    ws = sda.Workspace(p)
    seq = [dev(offsets([T // n_seq] * n_seq))] * 2
    seq[which] = dev(np.array([0, T] * 20 + [0], np.int32))
    o, lse = torch.full_like(q, 7.0), torch.full((T, 2), 7.0, device=DEV)
    sda.sda_prompt_attn_fwd(p, q, k, v, *seq, o, lse, ws.ptr, ws.nbytes)
    with pytest.raises(sda.SdaError) as e:
        ws.check()
    assert e.value.code == -3
    assert torch.all(o == 7) and torch.all(lse == 7)
    seq[which] = seq[1 - which]
    sda.sda_prompt_attn_fwd(p, q, k, v, *seq, o, lse, ws.ptr, ws.nbytes)
    ws.check()
    check_prompt(q, k, v, seq[0].cpu().numpy(), seq[1].cpu().numpy(), True, o, lse)


def test_cache_weights_of_a_prompts_last_rows_decide_its_first_eviction():
    """Whole prompts appended (weights zero), their last rows through cache attention, an eviction by those weights,
    then a token on the blocks that stayed: the order of calls that the header asks for."""
    rng = np.random.default_rng(38)
    H, H_kv, d, block, n, last, keep, recent = 8, 2, 64, 16, [150, 40, 300], 16, 64, 8
    c = Cache(rng, n, block, H, H_kv, d, n, extra=20, keep=keep, recent=recent)
    q, k, v = (bf16((sum(n), h, d), rng).to(DEV) for h in (H, H_kv, H_kv))
    O.append(f64(k), f64(v), c.seq, c.lens, c.table, block, c.host, c.w)
    c.append(k, v)
    c.ws.check()
    c.check_pool()
    assert np.array_equal(c.w_dev.cpu().numpy(), c.w)
    free = [b for b in range(c.n_blocks) if b not in c.table]
    wide = np.full((3, 5), -1, np.int32)                          # a block more than `keep` needs
    for b, t in enumerate(n):
        need = -(-(min(t, keep) + 1) // block)
        wide[b, :need], free = free[:need], free[need:]
    dst = np.ascontiguousarray(wide[:, :4])
    q_last = torch.cat([q[a - last:a] for a in c.seq[1:]])

    def call(table, rows):
        c.p = sda.cache_params(B=3, H=H, H_kv=H_kv, d=d, block=block, n_blocks=c.n_blocks, max_blocks=table.shape[1],
                               rows=3 * rows, max_new=rows, weights=True, keep=keep, recent=recent)
        c.ws, c.table, c.seq = sda.Workspace(c.p), table, offsets([rows] * 3)

    call(c.table, last)
    o = c.attend(q_last, c.w_dev, c.w_dev)
    c.ws.check()
    want, spread, wt = O.cache_attention(f64(q_last), c.seq, c.lens, c.table, block, c.host)
    size = max(score_size(f64(q_last), O.cache_values(c.host, "k", c.table[b], t, block, h))
               for b, t in enumerate(n) for h in range(H_kv))
    assert np.all(np.abs(f64(o) - want) <= attention_tolerance(want, spread, size, d, U_F16))
    got_w = c.w_dev.cpu().numpy()
    p_error = 2 * (2 * (d + 8) * U_F32 * size + 2.0 ** -20)
    for b, t in enumerate(n):
        i = np.arange(t)
        got = got_w[c.table[b, i // block], :, i % block].T
        assert np.all(np.abs(got - wt[b]) <= wt[b] * (p_error + (last * (H // H_kv) + 2) * U_F32))
    kept, m = torch.empty((3, H_kv, keep), dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    sda.sda_cache_evict(c.p, *c.args(), c.w_dev, dev(dst), kept, m, c.ws.ptr, c.ws.nbytes)
    c.ws.check()
    c.w = got_w
    want_kept, want_m = O.evict(c.lens, c.table, block, c.host, c.w, dst, keep, recent)
    assert np.array_equal(kept.cpu().numpy(), want_kept) and np.array_equal(m.cpu().numpy(), want_m)
    assert want_kept[0, 0, :keep - recent].max() >= keep - recent  # not merely the oldest: the weights decided
    c.check_pool()
    assert np.array_equal(c.w_dev.cpu().numpy(), c.w)
    call(wide, 1)
    c.lens = [int(x) + 1 for x in want_m]
    q1, k1, v1 = (bf16((3, h, d), rng).to(DEV) for h in (H, H_kv, H_kv))
    O.append(f64(k1), f64(v1), c.seq, c.lens, c.table, block, c.host, c.w)
    c.append(k1, v1)
    c.check_pool()
    check_cache_attention(c, q1)

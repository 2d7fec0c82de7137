"""Pins of the serving operators' oracle on the CPU: library attention, the library's 8-bit cast, counted facts."""
import numpy as np
import pytest
import torch

import oracle.serving as O

from _serving import make_pool, make_table, offsets


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_attention_is_library_attention(causal):
    rng = np.random.default_rng(1)
    H, H_kv, d = 4, 2, 16
    nq, nk = [5, 1, 7], [5, 3, 9]
    q, k, v = (rng.normal(size=(sum(n), h, d)) for n, h in ((nq, H), (nk, H_kv), (nk, H_kv)))
    sq, sk = offsets(nq), offsets(nk)
    o, lse, _ = O.prompt_attention(q, k, v, sq, sk, causal)
    for s in range(3):
        i, j = torch.arange(nq[s])[:, None], torch.arange(nk[s])[None]
        mask = (j <= i + nk[s] - nq[s]) if causal else torch.ones(nq[s], nk[s], dtype=torch.bool)
        t = lambda x, a: torch.from_numpy(x[a[s]:a[s + 1]]).transpose(0, 1)  # noqa: E731
        kk, vv = (t(x, sk).repeat_interleave(H // H_kv, 0) for x in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(t(q, sq), kk, vv, attn_mask=mask)
        assert np.allclose(o[sq[s]:sq[s + 1]], want.transpose(0, 1).numpy(), atol=1e-12)
        sc = (t(q, sq) @ kk.transpose(1, 2)) * d ** -0.5
        want = torch.logsumexp(sc.masked_fill(~mask, -torch.inf), -1)
        assert np.allclose(lse[sq[s]:sq[s + 1]], want.T.numpy(), atol=1e-12)


def test_rows_that_see_nothing():
    """More queries than keys under the causal mask: the first rows see no key."""
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(5, 1, 8)), rng.normal(size=(2, 1, 8)), rng.normal(size=(2, 1, 8))
    o, lse, _ = O.prompt_attention(q, k, v, [0, 5], [0, 2])
    assert np.all(o[:3] == 0) and np.all(lse[:3] == -np.inf)
    assert np.allclose(o[3, 0], v[0, 0]) and np.isfinite(lse[3:]).all()


def test_wanted_scale():
    for amax, s in ((448.0, 1.0), (448.0001, 2.0), (0.875, 2.0 ** -9), (0.876, 2.0 ** -8), (0.0, 2.0 ** -126),
                    (3.3e38, 2.0 ** 120)):
        assert O.wanted_scale(amax) == s
    for e in range(-30, 31):
        for m in (1.0, 1.2, 1.75, 1.76, 1.99):
            s = O.wanted_scale(m * 2.0 ** e)
            assert m * 2.0 ** e <= 448 * s and m * 2.0 ** e > 448 * s / 2


def test_append_in_pieces_keeps_the_values():
    """Tokens appended one by one hold, within half a step of the final scale's grid, what went in; growing the
    scale moves no value that stays normal."""
    rng = np.random.default_rng(3)
    H_kv, d, block, n = 2, 8, 16, 16
    x = rng.normal(size=(n, H_kv, d)) * np.exp2(np.arange(n) / 2)[:, None, None]
    x = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).double().numpy()
    pool = make_pool(rng, 2, H_kv, block, d)
    table = np.array([[1]], np.int32)
    for t in range(n):
        O.append(x[t:t + 1], x[t:t + 1], [0, 1], [t + 1], table, block, pool)
    for h in range(H_kv):
        assert pool["k_scale"][1, h] == O.wanted_scale(np.abs(x[:, h]).max())
        got = O.cache_values(pool, "k", table[0], n, block, h)
        scale = float(pool["k_scale"][1, h])
        step = np.maximum(np.abs(x[:, h]) / 8, scale * 2.0 ** -9)
        assert np.all(np.abs(got - x[:, h]) <= step)
        once = O.decode_e4m3(O.encode_e4m3((x[:, h] / scale).astype(np.float32))) * scale
        normal = np.abs(once) >= scale * 2.0 ** -6
        assert np.array_equal(got[normal], once[normal])


def test_cache_attention_is_prompt_attention_on_the_cache_values():
    rng = np.random.default_rng(4)
    H, H_kv, d, block = 4, 2, 16, 16
    lens, new = [37, 5, 16], [3, 5, 1]
    pool = make_pool(rng, 8, H_kv, block, d)
    table = make_table(rng, lens, block, 8)
    q = rng.normal(size=(sum(new), H, d))
    o, _, w = O.cache_attention(q, offsets(new), lens, table, block, pool)
    kv = [[np.concatenate([O.cache_values(pool, n, table[b], t, block, h)[:, None] for h in range(H_kv)], 1)
           for b, t in enumerate(lens)] for n in ("k", "v")]
    want, _, _ = O.prompt_attention(q, np.concatenate(kv[0]), np.concatenate(kv[1]), offsets(new), offsets(lens))
    assert np.allclose(o, want, atol=1e-12)
    for b in range(3):
        assert np.allclose(w[b].sum(), new[b] * H)


def test_kept_positions():
    assert O.kept_positions(np.array([1., 5, 5, 0, 2, 9]), 6, 4, 1).tolist() == [1, 2, 4, 5]
    assert O.kept_positions(np.array([5., 5, 5, 5]), 4, 2, 0).tolist() == [0, 1]      # ties to the lower
    assert O.kept_positions(np.array([0., -0.0, 0., 0]), 4, 3, 1).tolist() == [0, 1, 3]
    assert O.kept_positions(np.array([0., 1, np.nan, 3]), 4, 2, 0).tolist() == [2, 3]  # NaN counts as the largest
    assert O.kept_positions(np.array([np.inf, np.nan, 1]), 3, 1, 0).tolist() == [1]    # above infinity
    assert O.kept_positions(np.array([3., 2, 1]), 3, 8, 2).tolist() == [0, 1, 2]
    rng = np.random.default_rng(5)
    for _ in range(50):
        n, keep = rng.integers(1, 40, 2)
        recent = rng.integers(0, keep + 1)
        w = rng.integers(0, 6, n).astype(float)
        got = O.kept_positions(w, n, keep, recent)
        assert len(got) == min(n, keep) and np.all(np.diff(got) > 0)
        gone = np.setdiff1d(np.arange(n), got)
        older = got[got < n - min(recent, n)]
        assert all(w[g] < w[s] or (w[g] == w[s] and g > s) for g in gone for s in older)


def test_evict_moves_values():
    rng = np.random.default_rng(6)
    H_kv, d, block, lens, keep = 2, 8, 16, [50, 7], 20
    pool = make_pool(rng, 12, H_kv, block, d)
    table = make_table(rng, lens, block, 12)
    free = [b for b in range(12) if b not in table]
    dst = np.array([free[:2], [free[2], -1]], np.int32)
    w = rng.random((12, H_kv, block)).astype(np.float32)
    before = {n: [[O.cache_values(pool, n, table[b], t, block, h) for h in range(H_kv)] for b, t in enumerate(lens)]
              for n in ("k", "v")}
    kept, n = O.evict(lens, table, block, pool, w, dst, keep, 4)
    assert n.tolist() == [20, 7]
    for b in range(2):
        for h in range(H_kv):
            for name in ("k", "v"):
                got = O.cache_values(pool, name, dst[b], n[b], block, h)
                want = before[name][b][h][kept[b, h, :n[b]]]
                step = pool[name + "_scale"].max() * 2.0 ** -9   # only what becomes subnormal moves
                assert np.all(np.abs(got - want) <= step / 2)

"""Problems of the serving operators for the tests: seeded inputs on the host, a pool of blocks in shuffled order."""
import numpy as np
import torch

U_BF16, U_F16, U_F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24   # half a step, relative


def bf16(shape, rng, sd=1.0):
    return torch.from_numpy(rng.normal(0, sd, shape).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def offsets(lengths, first=0):
    return np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int32)


def make_pool(rng, n_blocks, H_kv, block, d, spread=3):
    """Codes of normal values, power-of-two scales over `spread` binades for each block and head."""
    pool = {}
    for n in ("k", "v"):
        x = torch.from_numpy(rng.normal(0, 64, (n_blocks, H_kv, block, d)).astype(np.float32)).clamp(-448, 448)
        pool[n + "_codes"] = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
        pool[n + "_scale"] = np.exp2(rng.integers(-7, -7 + spread, (n_blocks, H_kv))).astype(np.float32)
    return pool


def make_table(rng, lens, block, n_blocks, width=None, avoid=()):
    """Distinct random blocks for each sequence, -1 behind them."""
    need = [-(-int(t) // block) for t in lens]
    free = [b for b in rng.permutation(n_blocks) if b not in set(avoid)]
    table = np.full((len(lens), width or max(max(need), 1)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = free[at:at + n]
        at += n
    return table


def attention_tolerance(o, spread, score_size, d, u_p):
    """Bound of |o - o_exact| element by element.

    P is rounded once (u_p relative), the output once to bf16 (U_BF16). A score is a sum of d exact products in
    fp32, in any order: off by at most d U_F32 times the sum of their magnitudes, `score_size` (as a softmax
    argument), and a few roundings more for its scaling; tensor cores may drop bits instead of rounding, so twice
    that. The exponential's relative error is the score's absolute one, and it enters numerator and sum alike."""
    p_error = 2 * (2 * (d + 8) * U_F32 * score_size + 2.0 ** -20)
    return U_BF16 * np.abs(o) + (u_p + p_error) * spread * (1 + 2 * U_BF16) + 2.0 ** -120


def score_size(q, k, scale=None):
    """The largest sum of the products' magnitudes of a score: at most |q| |k| scale."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    return scale * np.linalg.norm(q, axis=-1).max() * np.linalg.norm(k, axis=-1).max()

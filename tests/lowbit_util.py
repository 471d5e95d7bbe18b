"""Plain forms of the 8-bit rows and the 4-bit weights, written from their
definitions (include/rom.h): element by element where a layout is concerned."""
import numpy as np
import torch

U = 2.0 ** -24  # unit roundoff of float32


def half_step(dtype) -> float:
    """Largest rounding error of a normal value, relative to it."""
    return torch.finfo(dtype).eps / 2


def gamma(n: int, u: float = U) -> float:
    return n * u / (1.0 - n * u)


def rows_to_8bit(v: torch.Tensor):
    """float32 rows -> (e4m3 codes, float32 scales), in the definition's own
    float32 operations (each of them rounded to nearest), so that the kernels'
    codes have to be these."""
    v = v.float().cpu()
    a = v.abs().amax(-1).clamp(min=2.0 ** -100)
    inv = torch.tensor(448.0) / a
    scaled = (v * inv.unsqueeze(-1)).clamp(-448.0, 448.0)  # 448 (1 + 2^-22) rounds to 448
    return scaled.to(torch.float8_e4m3fn), a / torch.tensor(448.0)


def w4_position(N, K):
    """For every (n, c): the byte of q (within an expert) and the nibble's shift."""
    kb = -(-K // 128)
    n, c = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    r, cc = n % 16, c % 128
    h, g = r // 8, r % 8
    i, a, t, b, d = cc // 32, cc // 16 % 2, cc // 4 % 4, cc // 2 % 2, cc % 2
    p = 4 * d + 2 * a + b
    byte = ((n // 16) * kb + c // 128) * 1024 + h * 512 + (4 * g + t) * 16 + i * 4 + p // 2
    return byte, 4 * (p % 2)


def w4_decode(q, s, N, K):
    """Codes uint8 and scales bf16 (tensors in the library's storage) -> float64
    [E, N, K] values."""
    E, _, kb = q.shape[:3]
    group = 128 // s.shape[-1]
    byte, shift = w4_position(N, K)
    flat = q.cpu().numpy().reshape(E, -1)
    codes = (flat[:, byte] >> shift) & 15
    sf = s.float().cpu().numpy().astype(np.float64)  # [E, Nt, Kb, 16, G]
    n, c = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    scale = sf[:, n // 16, c // 128, n % 16, c % 128 // group]
    return (codes.astype(np.float64) - 8.0) * scale, codes, scale


def make_routing(T, E, k, seed, pin=None):
    """Distinct experts per token, positive weights, and the expert order."""
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32).reshape(T, k)
    if pin is not None:
        idx[:, 0] = pin
    w = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    flat = idx.reshape(-1)
    order = np.argsort(flat, kind="stable").astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]).astype(np.int32)
    return idx, w, order, off

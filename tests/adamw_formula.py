"""The 8-bit moments of an AdamW step in plain fp32 arithmetic, on the CPU: codes, scales and what is kept beside the codes. numpy's
products, sums, quotients and roots are each rounded correctly (torch's root on the CPU is one unit off for one value in 160)."""
import numpy as np
import torch

F, U = np.float32, np.uint32
BLOCK = 128


def _fp8(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=F)).to(torch.float8_e4m3fn)


def _power(value):
    """2^e of codes' values, 2^-6 at least: the step between codes is an eighth of it."""
    return np.maximum(value.view(U) & U(0x7F800000), U(0x3C800000)).view(F)


def dither(e, step, m):
    """32 bits for each element: the low 16 for the rounding of m, the high 16 for that of sqrt(v)."""
    e, step = np.asarray(e, dtype=np.uint64), int(step)
    low, high = (e & np.uint64(0xFFFFFFFF)).astype(U), (e >> np.uint64(32)).astype(U)
    with np.errstate(over="ignore"):
        seed = U(step * 0xB5297A4D & 0xFFFFFFFF) + high * U(0x68E31DA5)
        x = (low * U(0x9E3779B1) + seed) ^ m.view(U)
        x = (x ^ x >> U(15)) * U(0xD1B54A33)
        x = (x ^ x >> U(13)) * U(0x8CB92BA7)
    return x ^ x >> U(16)


def encode(x, random):
    """(codes, scales, k) of whole blocks; `random`: 16 bits for each element, or None for codes alone (k 0)."""
    x = x.reshape(-1, BLOCK)
    most = np.maximum(np.abs(x).max(axis=1), F(2.0 ** -100))
    c = np.clip(x * (F(448) * (F(1) / most))[:, None], F(-448), F(448)).astype(F).reshape(-1)
    codes = _fp8(c)
    if random is None:
        k = np.zeros(c.shape, dtype=np.int32)
    else:
        value = codes.float().numpy()
        steps = (c - value) * (F(112) / _power(value))
        k = np.floor(steps + random.astype(F) * F(2.0 ** -16)).astype(np.int32)
    return codes.view(torch.uint8).numpy(), (most / F(448)).astype(F), k


def decode(codes, scales, k):
    value = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    x = value + k.astype(F) * (_power(value) * F(1.0 / 112.0))
    return (x.reshape(-1, BLOCK) * scales[:, None]).reshape(-1)


def low(fine):
    n = (fine & 15).astype(np.int32)
    return n - 16 * (n > 7)


class Moments:
    """Moments of one tensor of n elements, as the state keeps them."""

    def __init__(self, n, keep=True):
        whole = -(-n // BLOCK) * BLOCK
        self.n, self.keep, self.start = n, keep, 0  # start: the first element's place in its tensor
        self.m, self.v, self.fine = (np.zeros(whole, dtype=np.uint8) for _ in range(3))
        self.m_scale, self.v_scale = (np.zeros(whole // BLOCK, dtype=F) for _ in range(2))

    def values(self):
        """(m, sqrt(v)) in whole blocks."""
        return decode(self.m, self.m_scale, low(self.fine)), decode(self.v, self.v_scale, low(self.fine >> 4))

    def step(self, g, number, betas):
        m, r = self.values()
        wide = np.zeros(m.shape, dtype=F)
        wide[:self.n] = g
        m = m * F(betas[0]) + wide * F(1.0 - betas[0])
        v = (r * r) * F(betas[1]) + (wide * wide) * F(1.0 - betas[1])
        root = np.sqrt(v)
        m[self.n:] = root[self.n:] = 0
        random = dither(np.arange(self.start, self.start + m.size), number, m) if self.keep else None
        self.m, self.m_scale, km = encode(m, random & U(0xFFFF) if self.keep else None)
        self.v, self.v_scale, kv = encode(root, random >> U(16) if self.keep else None)
        self.fine = ((km & 15) | (kv & 15) << 4).astype(np.uint8)

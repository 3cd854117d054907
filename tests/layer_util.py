"""References of the 4-bit operands for the tests of a layer's operators, on the host in numpy,
where frexp and ldexp are exact."""
import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def nearest_e2m1(a):
    """Code (0 to 7) of each magnitude: nearest value, ties to the even code, 6 from there on."""
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.zeros(a.shape, np.int64)
    for i, m in enumerate(mid):  # between codes i and i + 1: a tie goes to the even one
        code += (a > m) | ((a == m) & (i % 2 == 1))
    return code


def micro_ref(x):
    """(codes (rows, K) with the sign as 8, scale bytes (rows, K / 32)) of finite rows."""
    v = x.double().cpu().numpy()
    b = v.reshape(v.shape[0], -1, 32)
    m, e = np.frexp(np.abs(b).max(-1))  # m * 2^e, m from 0.5 on
    byte = np.where(m > 0, np.maximum(e - 1 - 2 + (m >= 0.875) + 127, 0), 0).astype(np.int64)
    code = nearest_e2m1(np.abs(b) / np.ldexp(1.0, byte - 127)[..., None])
    return (code + 8 * np.signbit(b)).reshape(v.shape), byte


def packed(codes):
    """Two codes a byte, the first low."""
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).astype(np.uint8)


def row_words(byte):
    """Scale bytes (rows, K / 32) as (ceil(K / 128), rows, 4)."""
    rows, nb = byte.shape
    out = np.zeros((rows, -(-nb // 4) * 4), np.uint8)
    out[:, :nb] = byte
    return np.ascontiguousarray(out.reshape(rows, -1, 4).transpose(1, 0, 2))


def weight_pieces(byte):
    """Scale bytes (E, N, K / 32) as (E, ceil(N / 128), ceil(K / 128), 32, 4, 4)."""
    E, N, nb = byte.shape
    out = np.zeros((E, -(-N // 128) * 128, -(-nb // 4) * 4), np.uint8)
    out[:, :N, :nb] = byte
    return np.ascontiguousarray(out.reshape(E, out.shape[1] // 128, 4, 32, -1, 4).transpose(0, 1, 4, 3, 2, 5))


def code_values(q):
    """Values in units of their scales of packed codes (..., K / 2): (..., K) float64."""
    table = torch.tensor(np.concatenate([E2M1, -E2M1]), device=q.device)
    return torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).flatten(-2)


def scale_values(byte):
    """2^(byte - 127) in 64 bits, NaN for 255."""
    v = torch.exp2(byte.double() - 127)
    return torch.where(byte == 255, torch.full_like(v, float("nan")), v)


def row_values(q, s):
    """What rows' codes and scales stand for, in 64 bits."""
    K = q.shape[1] * 2
    byte = s.view(torch.uint8).permute(1, 0, 2).flatten(1)[:, :K // 32]
    return code_values(q) * scale_values(byte).repeat_interleave(32, 1)


def weight_values(q, s):
    """What weights' codes and scales stand for, in 64 bits: (E, N, K)."""
    E, N, K = q.shape[0], q.shape[1], q.shape[2] * 2
    b = s.view(torch.uint8)
    byte = b.permute(0, 1, 4, 3, 2, 5).reshape(E, b.shape[1] * 128, -1)[:, :N, :K // 32]
    return code_values(q) * scale_values(byte).repeat_interleave(32, 2)

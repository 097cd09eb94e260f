"""fp64 reference of the microscaled 4-bit code and product (numpy, no code shared with the library).

Definitions as in include/muon.h: muon_mx4_quantize, muon_mx4_matmul."""
import numpy as np

BLOCK, UNIT = 32, 128
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_bytes(blocks):
    """Scale bytes of float64 blocks (last axis = the block)."""
    top = np.abs(blocks).max(-1)
    bad = ~np.isfinite(top)
    with np.errstate(divide="ignore", invalid="ignore"):
        _, e = np.frexp(np.where(bad, 1.0, top))  # top = f 2^e, f in [1/2, 1): its own exponent is e - 1
    byte = np.where(top == 0, 0, np.maximum(e - 1 - 2 + 127, 0))
    return np.where(bad, 255, byte).astype(np.uint8)


def quantize(X):
    """(codes, scales) of a 2-D float64 matrix along its rows, in the library's layout."""
    rows, cols = X.shape
    units = -(-cols // UNIT)
    P = np.zeros((rows, units * UNIT))
    P[:, :cols] = X
    B = P.reshape(rows, units * 4, BLOCK)
    byte = scale_bytes(B)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.abs(B) * np.ldexp(1.0, 127 - byte.astype(np.int64))[..., None]
        y = np.where(byte[..., None] == 255, 0.0, np.minimum(y, 6.0))
    dist = np.abs(y[..., None] - MAGNITUDES)
    best = dist.min(-1, keepdims=True)
    level = np.argmax(dist == best, -1)                         # the lower one of two equally near
    tie = (dist == best).sum(-1) > 1
    level = np.where(tie & (level % 2 == 1), level + 1, level)  # ties to the even code
    code = level | np.where(np.signbit(B) & (byte[..., None] != 255), 8, 0)
    code = code.reshape(rows, units, UNIT).astype(np.uint8)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    return packed.transpose(1, 0, 2).copy(), byte.reshape(rows, units, 4).transpose(1, 0, 2).copy()


def decode(codes, scales, cols):
    """float64 values of codes/scales in the library's layout (NaN where the scale byte is 255)."""
    units, rows, _ = codes.shape
    c = codes.transpose(1, 0, 2).reshape(rows, units * 64)
    nib = np.empty((rows, units * UNIT), dtype=np.int64)
    nib[:, 0::2] = c & 15
    nib[:, 1::2] = c >> 4
    value = MAGNITUDES[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    byte = scales.transpose(1, 0, 2).reshape(rows, units * 4).astype(np.int64)
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    return (value.reshape(rows, units * 4, BLOCK) * s[..., None]).reshape(rows, units * UNIT)[:, :cols]


def matmul(A, B):
    """A B^T of decoded float64 matrices and the bound of its fp32 rounding: every product is exact in fp32 (two 2-bit
    significands and a power of two), each of the k additions rounds the running sum by at most a step, 2^-23 of the
    sum of magnitudes."""
    return A @ B.T, (A.shape[1] + 2) * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T)

"""Helpers of the GPU tests of the norm, routing from scores and rows in 8 bits."""
import numpy as np

from oracle import front_oracle as F

BLOCKS = (16, 32, 64, 128)


def code_bytes(torch, codes):
    return codes.view(torch.uint8).cpu().numpy()


def stored(torch, codes, scales, block):
    """The values that codes and scales stand for, by the oracle."""
    fmt = "int8" if codes.dtype == torch.uint8 else "e4m3"
    return F.values(code_bytes(torch, codes), scales.double().cpu().numpy(), fmt, block)


def check_eight(torch, codes, scales, block, ref, e, label):
    """Codes and scales hold a row whose elements lie within e of ref: every scale is the least of a largest magnitude
    within the block's errors, every value within half a step of the element (a power of two, or 2^-4 of the value but
    at least the subnormal half step 2^-10 of the scale)."""
    fmt = "int8" if codes.dtype == torch.uint8 else "e4m3"
    got, s = stored(torch, codes, scales, block), scales.double().cpu().numpy()
    M, N = ref.shape
    e = np.broadcast_to(e, ref.shape)
    for b in range(s.shape[1]):
        part = slice(b * block, min(N, (b + 1) * block))
        a, ea = np.abs(ref[:, part]), e[:, part]
        lo, hi = np.maximum((a - ea).max(1), 0), (a + ea).max(1)
        for m in range(M):
            x, y = (2.0 ** F.scale_exponent(v, fmt) for v in (lo[m], hi[m]))
            # (a largest magnitude that may be 0: any scale up to y, or 1)
            assert x <= s[m, b] <= y or (lo[m] == 0 and s[m, b] == 1.0), (label, m, b, s[m, b], x, y)
    step = np.repeat(s, block, axis=1)[:, :N]
    half = step / 2 if fmt == "int8" else np.maximum((np.abs(ref) + e) * 2.0 ** -4, step * 2.0 ** -10)
    err = np.abs(got - ref)
    assert (err <= half + e).all(), (label, float((err / (half + e)).max()))

"""How the library tiles a stored-weight product, read from its host-side plan (not collected
by pytest; needs no GPU)."""

import ctypes

import bit_quantized_mixture_nf4_amd as e4b
from bit_quantized_mixture_nf4_amd import _lib

ROWS, T128, TALL, T256 = 0, 1, 2, 3  # few rows, 128 x 128, 256 x 128, 256 x 256


def linear_plan(E, rows, inn, out, codebook="nf4"):
    """(forward tiles, gradient tiles, forward shares of k, gradient shares of k); the status if refused."""
    plan = e4b.load()._ZN3e4b11plan_linearEPK9e4b_stackliiPNS_10LinearPlanE  # e4b::plan_linear
    plan.restype = ctypes.c_int32
    plan.argtypes = [ctypes.POINTER(_lib.E4bStack), ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p]
    fake = 0x10000  # never read here
    mx = codebook == "mxfp4"
    st = _lib.E4bStack(fake, fake, E, out, inn, 32 if mx else 64, e4b.CODEBOOKS[codebook], fake)
    p = (ctypes.c_int32 * 128)()  # the plan begins with these four
    status = plan(ctypes.byref(st), rows, _lib.E4B_ACT_NONE, _lib.E4B_BF16, p)
    return status if status != _lib.E4B_OK else tuple(p[:4])

"""Argument types of the serving operators' C functions (include/kda.h)."""
import ctypes

_VP, _I64, _F32, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int

_STEP = [_VP] * 5 + [_F32] + [_VP] * 3 + [_F32, _VP, _I32, _I64, _VP, _VP] + [_I64] * 3
_LA_STEP = ([_VP, _I64] * 3 + [_VP, _VP, _F32, _VP, _VP, _I32, _I64, _VP, _VP] + [_I64] * 4)
_LA_FWD = ([_VP, _I64] * 3 + [_VP, _VP, _F32, _VP, _VP, _I32, _VP, _I32, _VP] + [_I64] * 7
           + [_VP, _I64])
_ATTN_FWD = ([_VP, _I64] * 3 + [_F32] + [_VP] * 5 + [_I64] * 9 + [_VP, _I64])


def declare(lib) -> None:
    """Sets the argument types of the serving operators' C functions, and their addresses
    (``name_at``) for the compiled calls."""
    for name, args in (("kda_step", _STEP), ("kda_la_step", _LA_STEP),
                       ("kda_la_fwd", _LA_FWD), ("kda_attn_fwd", _ATTN_FWD)):
        getattr(lib, name).argtypes = args + [_VP]
        getattr(lib, name).restype = _I32
        setattr(lib, name + "_at", ctypes.cast(getattr(lib, name), _VP).value)
        getattr(lib, name + "_check").argtypes = args
        getattr(lib, name + "_check").restype = _I32
    for name in ("kda_la_workspace_bytes", "kda_attn_workspace_bytes"):
        setattr(lib, name + "_at", ctypes.cast(getattr(lib, name), _VP).value)
    lib.kda_la_workspace_bytes.argtypes = [_I64] * 5
    lib.kda_la_workspace_bytes.restype = _I64
    lib.kda_attn_workspace_bytes.argtypes = [_I64] * 9
    lib.kda_attn_workspace_bytes.restype = _I64

"""fp64 CPU attention oracle -- TEST INFRASTRUCTURE ONLY.

Only the test suite, the smoke check and the benchmark's CPU-baseline /
reference arm may import this package.  The product library never does, and
this package imports nothing from it: the two share no code.

The arithmetic lives in ``attn_oracle.c`` (plain C, fp64, one materialised
probability row per query); this module compiles it with gcc and marshals
numpy arrays through ctypes.  Every function here follows the definition
written at the top of ``attn_oracle.c``, which cites the pages it restates:

* ferrotensor_backend engine/attention.rs -- AttentionOptions (causal offset,
  window predicate), AttentionDims (head_dim, GQA divisibility, 1/sqrt(hd)).
* brotensor ops/flash_attention.h -- key mask (> 0.5 keeps a key), softcap
  position, GQA head map, decode row positions, overwrite semantics.
* vision_rs flash_attn2.rs -- forward with saved log-sum-exp, dQ and dK/dV.
* forge attention.metal -- unfused forward with materialised P, D = dO.O,
  softcap derivative, GQA group sums in dK/dV.

Pins: every function here is checked against closed forms, invariants, an
independent torch fp64 route and finite differences in
``tests/test_oracle_pins.py``.  One reading is a choice among conflicting
pages rather than a fixed fact: the non-causal sliding window (ferrotensor's
``|p - j| < window``); its implementation is pinned to that formula, the choice
of formula is recorded as a reading.
"""
from __future__ import annotations

import ctypes
import os
import subprocess
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_SRC = os.path.join(_HERE, "attn_oracle.c")
_BUILD = os.path.join(_HERE, "_build")
_LIB_PATH = os.path.join(_BUILD, "liboracle.so")
_lock = threading.Lock()
_lib = None


def build(force: bool = False) -> str:
    """Compile attn_oracle.c into a shared library (gcc, OpenMP). Returns its path."""
    os.makedirs(_BUILD, exist_ok=True)
    stale = (not os.path.exists(_LIB_PATH)) or os.path.getmtime(_LIB_PATH) < os.path.getmtime(_SRC)
    if force or stale:
        tmp = _LIB_PATH + ".tmp.%d" % os.getpid()
        cmd = ["gcc", "-O2", "-fPIC", "-shared", "-fopenmp", "-std=c99", _SRC, "-o", tmp, "-lm"]
        subprocess.run(cmd, check=True)
        os.replace(tmp, _LIB_PATH)
    return _LIB_PATH


def _load():
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        lib = ctypes.CDLL(build())
        dp = ctypes.POINTER(ctypes.c_double)
        common = [ctypes.c_int] * 6 + [ctypes.c_double, ctypes.c_int, ctypes.c_int, ctypes.c_double,
                                       ctypes.c_longlong, dp, ctypes.c_longlong]
        lib.oracle_attn_fwd.argtypes = [dp, dp, dp, dp, dp] + common
        lib.oracle_attn_fwd.restype = ctypes.c_int
        lib.oracle_attn_probs.argtypes = [dp, dp, dp, dp, ctypes.c_int, ctypes.c_int] + common
        lib.oracle_attn_probs.restype = ctypes.c_int
        lib.oracle_attn_bwd.argtypes = [dp] * 7 + common
        lib.oracle_attn_bwd.restype = ctypes.c_int
        llp = ctypes.POINTER(ctypes.c_longlong)
        common_ex = [ctypes.c_int] * 6 + [ctypes.c_double, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_double,
                                          ctypes.c_longlong, dp, ctypes.c_longlong, dp, llp]
        lib.oracle_attn_fwd_ex.argtypes = [dp, dp, dp, dp, dp] + common_ex
        lib.oracle_attn_fwd_ex.restype = ctypes.c_int
        lib.oracle_attn_probs_ex.argtypes = [dp, dp, dp, dp, ctypes.c_int, ctypes.c_int] + common_ex
        lib.oracle_attn_probs_ex.restype = ctypes.c_int
        lib.oracle_attn_bwd_ex.argtypes = [dp] * 7 + common_ex
        lib.oracle_attn_bwd_ex.restype = ctypes.c_int
        lib.oracle_num_threads.argtypes = []
        lib.oracle_num_threads.restype = ctypes.c_int
        _lib = lib
        return lib


def _f64(a):
    return np.ascontiguousarray(np.asarray(a, dtype=np.float64))


def _ptr(a):
    if a is None:
        return None
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_double))


def _shapes(q, k, H, Hkv):
    if q.ndim != 3 or k.ndim != 3:
        raise ValueError("q must be [B,Tq,H*hd] and k/v [B,Tk,Hkv*hd]")
    B, Tq, qc = q.shape
    _, Tk, kc = k.shape
    if qc % H or kc % Hkv or qc // H != kc // Hkv:
        raise ValueError("inconsistent head sizes")
    return B, Tq, Tk, qc // H


def _mask(key_mask, B, Tk):
    """Returns (array or None, batch stride). A 1-D mask is shared by every batch."""
    if key_mask is None:
        return None, 0
    m = _f64(key_mask)
    if m.ndim == 1:
        if m.shape[0] != Tk:
            raise ValueError("key mask must have Tk entries")
        return m, 0
    if m.shape != (B, Tk):
        raise ValueError("key mask must be [Tk] or [B,Tk]")
    return m, Tk


def _common(B, Tq, Tk, H, Hkv, hd, scale, causal, window, softcap, q_offset, m, ms):
    return [B, Tq, Tk, H, Hkv, hd, float(scale), int(bool(causal)), int(window), float(softcap),
            int(q_offset), _ptr(m), int(ms)]


def num_threads() -> int:
    """OpenMP threads the oracle runs on."""
    return int(_load().oracle_num_threads())


def fwd(q, k, v, *, H, Hkv, scale, causal=False, window=0, softcap=0.0, q_offset=0,
        key_mask=None):
    """O [B,Tq,H*hd] and LSE [B,H,Tq] of the plain definition (fp64)."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Tq, Tk, hd = _shapes(q, k, H, Hkv)
    m, ms = _mask(key_mask, B, Tk)
    o = np.zeros((B, Tq, H * hd), np.float64)
    lse = np.zeros((B, H, Tq), np.float64)
    rc = _load().oracle_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                 *_common(B, Tq, Tk, H, Hkv, hd, scale, causal, window, softcap,
                                          q_offset, m, ms))
    if rc != 0:
        raise ValueError("oracle_attn_fwd rejected its arguments")
    return o, lse


def probs(q, k, v, b, h, *, H, Hkv, scale, causal=False, window=0, softcap=0.0, q_offset=0,
          key_mask=None):
    """The materialised probability matrix P [Tq,Tk] of batch b, head h."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Tq, Tk, hd = _shapes(q, k, H, Hkv)
    m, ms = _mask(key_mask, B, Tk)
    P = np.zeros((Tq, Tk), np.float64)
    rc = _load().oracle_attn_probs(_ptr(q), _ptr(k), _ptr(v), _ptr(P), int(b), int(h),
                                   *_common(B, Tq, Tk, H, Hkv, hd, scale, causal, window, softcap,
                                            q_offset, m, ms))
    if rc != 0:
        raise ValueError("oracle_attn_probs rejected its arguments")
    return P


def bwd(q, k, v, do, *, H, Hkv, scale, causal=False, window=0, softcap=0.0, q_offset=0,
        key_mask=None):
    """dQ, dK, dV of the plain definition, with P rebuilt from the inputs."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    B, Tq, Tk, hd = _shapes(q, k, H, Hkv)
    if do.shape != q.shape:
        raise ValueError("dO must have q's shape")
    m, ms = _mask(key_mask, B, Tk)
    dq = np.zeros_like(q)
    dk = np.zeros_like(k)
    dv = np.zeros_like(v)
    rc = _load().oracle_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                                 *_common(B, Tq, Tk, H, Hkv, hd, scale, causal, window, softcap,
                                          q_offset, m, ms))
    if rc != 0:
        raise ValueError("oracle_attn_bwd rejected its arguments")
    return dq, dk, dv


def _bias(bias, B, H, Tq, Tk):
    """(array or None, 4 strides): an additive bias broadcastable to [B, H, Tq, Tk],
    size-1 dimensions read with stride 0 (ferrotensor engine/attention.rs, mask_strides)."""
    if bias is None:
        return None, None
    a = _f64(bias)
    if a.ndim != 4:
        raise ValueError("bias must be 4-D [B|1, H|1, Tq|1, Tk|1]")
    full = (B, H, Tq, Tk)
    st = []
    for dim, n, sb in zip(a.shape, full, a.strides):
        if dim not in (1, n):
            raise ValueError("bias shape %s does not broadcast to %s" % (a.shape, full))
        st.append(0 if dim == 1 else sb // 8)
    return a, (ctypes.c_longlong * 4)(*st)


def _common_ex(B, Tq, Tk, H, Hkv, hd, scale, wl, wr, softcap, q_offset, m, ms, bias, bs):
    return [B, Tq, Tk, H, Hkv, hd, float(scale), int(wl), int(wr), float(softcap), int(q_offset), _ptr(m), int(ms),
            _ptr(bias), bs]


def fwd_ex(q, k, v, *, H, Hkv, scale, window_left=-1, window_right=-1, softcap=0.0, q_offset=0, key_mask=None,
           bias=None):
    """O and LSE with the two-sided window [p - window_left, p + window_right]
    (negative = unbounded) and an optional additive bias (see attn_oracle.c)."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Tq, Tk, hd = _shapes(q, k, H, Hkv)
    m, ms = _mask(key_mask, B, Tk)
    bb, bs = _bias(bias, B, H, Tq, Tk)
    o = np.zeros((B, Tq, H * hd), np.float64)
    lse = np.zeros((B, H, Tq), np.float64)
    rc = _load().oracle_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                    *_common_ex(B, Tq, Tk, H, Hkv, hd, scale, window_left, window_right, softcap,
                                                q_offset, m, ms, bb, bs))
    if rc != 0:
        raise ValueError("oracle_attn_fwd_ex rejected its arguments")
    return o, lse


def probs_ex(q, k, v, b, h, *, H, Hkv, scale, window_left=-1, window_right=-1, softcap=0.0, q_offset=0,
             key_mask=None, bias=None):
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, Tq, Tk, hd = _shapes(q, k, H, Hkv)
    m, ms = _mask(key_mask, B, Tk)
    bb, bs = _bias(bias, B, H, Tq, Tk)
    P = np.zeros((Tq, Tk), np.float64)
    rc = _load().oracle_attn_probs_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(P), int(b), int(h),
                                      *_common_ex(B, Tq, Tk, H, Hkv, hd, scale, window_left, window_right, softcap,
                                                  q_offset, m, ms, bb, bs))
    if rc != 0:
        raise ValueError("oracle_attn_probs_ex rejected its arguments")
    return P


def bwd_ex(q, k, v, do, *, H, Hkv, scale, window_left=-1, window_right=-1, softcap=0.0, q_offset=0, key_mask=None,
           bias=None):
    """dQ, dK, dV of fwd_ex (the bias is a constant: it enters through P only)."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    B, Tq, Tk, hd = _shapes(q, k, H, Hkv)
    m, ms = _mask(key_mask, B, Tk)
    bb, bs = _bias(bias, B, H, Tq, Tk)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    rc = _load().oracle_attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                                    *_common_ex(B, Tq, Tk, H, Hkv, hd, scale, window_left, window_right, softcap,
                                                q_offset, m, ms, bb, bs))
    if rc != 0:
        raise ValueError("oracle_attn_bwd_ex rejected its arguments")
    return dq, dk, dv


def varlen_fwd(q, k, v, cu_q, cu_k, *, H, Hkv, scale, causal=False, window=0, softcap=0.0):
    """Packed variable-length forward (brotensor ops/flash_attention.h,
    flash_attention_varlen_forward): sequence b is rows cu_q[b] .. cu_q[b+1]-1 of
    q [total_q, H*hd] and rows cu_k[b] .. cu_k[b+1]-1 of k/v, attended to as its
    own batch of one with query positions counted from its first row; nothing
    crosses sequences.  Returns O [total_q, H*hd] (zero on rows outside every
    sequence) and LSE as a list of [H, Tq_b] arrays, one per sequence."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    hd = q.shape[1] // H
    o = np.zeros_like(q)
    lses = []
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        if q1 == q0:
            lses.append(np.zeros((H, 0)))
            continue
        if k1 == k0:  # no key at all: every row fully masked (O = 0, LSE = -inf)
            lses.append(np.full((H, q1 - q0), -np.inf))
            continue
        ob, lb = fwd(q[None, q0:q1], k[None, k0:k1], v[None, k0:k1], H=H, Hkv=Hkv, scale=scale, causal=causal,
                     window=window, softcap=softcap)
        o[q0:q1] = ob[0]
        lses.append(lb[0])
    return o, lses


def varlen_bwd(q, k, v, do, cu_q, cu_k, *, H, Hkv, scale, causal=False, window=0, softcap=0.0):
    """Backward of varlen_fwd (brotensor flash_attention_varlen_backward: the
    per-sequence backward; excluded positions contribute nothing).  Returns dQ,
    dK, dV on the packed rows, zero outside every sequence."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        if q1 == q0 or k1 == k0:
            continue
        gq, gk, gv = bwd(q[None, q0:q1], k[None, k0:k1], v[None, k0:k1], do[None, q0:q1], H=H, Hkv=Hkv, scale=scale,
                         causal=causal, window=window, softcap=softcap)
        dq[q0:q1], dk[k0:k1], dv[k0:k1] = gq[0], gk[0], gv[0]
    return dq, dk, dv


def rope(x, *, head_dim, pos=0, theta=10000.0):
    """Rotate-half rotary embedding (ferrotensor engine/attention.rs, rope /
    rope_theta): x is [batch, seq, heads*head_dim]; every head vector of token s
    (counted within its sequence) gets position pos + s, and its pair
    (x[i], x[i + head_dim/2]), i < head_dim/2, turns by the angle
    (pos + s) * theta**(-2i/head_dim):
        x'[i]          = x[i] cos - x[i + head_dim/2] sin
        x'[i + hd/2]   = x[i + head_dim/2] cos + x[i] sin
    Returns a new fp64 array (the page rotates in place)."""
    x = _f64(x)
    B, T, C = x.shape
    hd = int(head_dim)
    if hd % 2 or C % hd:
        raise ValueError("head_dim must be even and divide the row")
    half = hd // 2
    out = x.copy().reshape(B, T, C // hd, hd)
    xin = x.reshape(B, T, C // hd, hd)
    for s in range(T):
        p = float(pos + s)
        for i in range(half):
            ang = p * float(theta) ** (-2.0 * i / hd)
            c, sn = np.cos(ang), np.sin(ang)
            a, b = xin[:, s, :, i], xin[:, s, :, i + half]
            out[:, s, :, i] = a * c - b * sn
            out[:, s, :, i + half] = b * c + a * sn
    return out.reshape(B, T, C)


def _packed_rows(seq_bounds, L, window):
    """Visible keys of every row of a packed fused-QKV batch: row r attends keys j of
    its own sequence, seq_bounds[r, 0] <= j < seq_bounds[r, 1], and with window > 0
    only those with |r - j| <= window // 2 (brotensor ops/flash_attention.h,
    flash_attention_packed_qkv_forward)."""
    sb = np.asarray(seq_bounds, dtype=np.int64).reshape(L, 2)
    rows = []
    for r in range(L):
        j = np.arange(max(int(sb[r, 0]), 0), min(int(sb[r, 1]), L))
        if window > 0:
            j = j[np.abs(r - j) <= window // 2]
        rows.append(j)
    return rows


def _split_qkv(qkv, H):
    qkv = _f64(qkv)
    L, C = qkv.shape
    hd = C // (3 * H)
    if 3 * H * hd != C:
        raise ValueError("qkv rows must hold 3 * H * head_dim values")
    return (qkv[:, :H * hd].reshape(L, H, hd), qkv[:, H * hd:2 * H * hd].reshape(L, H, hd),
            qkv[:, 2 * H * hd:].reshape(L, H, hd), L, hd)


def packed_qkv_fwd(qkv, seq_bounds, *, H, scale, window=0):
    """Packed bidirectional self-attention straight off a fused QKV projection
    (brotensor ops/flash_attention.h, flash_attention_packed_qkv_forward): qkv is
    [L, 3*H*hd], each row [q heads | k heads | v heads]; the visible keys of row r
    are those of _packed_rows.  Written out row by row in numpy fp64 (independent of
    attn_oracle.c).  Returns O [L, H*hd] and LSE [H, L] (-inf for a row that sees
    no key, whose O is 0)."""
    q, k, v, L, hd = _split_qkv(qkv, H)
    o = np.zeros((L, H, hd))
    lse = np.full((H, L), -np.inf)
    for r, j in enumerate(_packed_rows(seq_bounds, L, window)):
        if j.size == 0:
            continue
        s = scale * np.einsum("hd,jhd->hj", q[r], k[j])  # [H, keys]
        mx = s.max(axis=1, keepdims=True)
        p = np.exp(s - mx)
        l = p.sum(axis=1, keepdims=True)
        o[r] = np.einsum("hj,jhd->hd", p / l, v[j])
        lse[:, r] = (mx + np.log(l))[:, 0]
    return o.reshape(L, H * hd), lse


def packed_qkv_bwd(qkv, do, seq_bounds, *, H, scale, window=0):
    """Backward of packed_qkv_fwd (brotensor flash_attention_packed_qkv_backward):
    dQKV [L, 3*H*hd], each row [dQ heads | dK heads | dV heads].  Per row r and head:
    P = softmax(scale * q_r . k_j) over its visible keys, dP_j = dO_r . v_j,
    dS = P (dP - sum(P dP)), dq_r = scale * sum_j dS_j k_j, dk_j += scale * dS_j q_r,
    dv_j += P_j dO_r; row by row in numpy fp64."""
    q, k, v, L, hd = _split_qkv(qkv, H)
    do = _f64(do).reshape(L, H, hd)
    dq, dk, dv = np.zeros((L, H, hd)), np.zeros((L, H, hd)), np.zeros((L, H, hd))
    for r, j in enumerate(_packed_rows(seq_bounds, L, window)):
        if j.size == 0:
            continue
        s = scale * np.einsum("hd,jhd->hj", q[r], k[j])
        p = np.exp(s - s.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        dp = np.einsum("hd,jhd->hj", do[r], v[j])
        ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
        dq[r] = scale * np.einsum("hj,jhd->hd", ds, k[j])
        dk[j] += scale * np.einsum("hj,hd->jhd", ds, q[r])
        dv[j] += np.einsum("hj,hd->jhd", p, do[r])
    return np.concatenate([dq.reshape(L, -1), dk.reshape(L, -1), dv.reshape(L, -1)], axis=1)


def turn_part(x, pos, *, H, inv_freq, start=0, interleaved=False, amplitude=1.0, backward=False):
    """Rows x [n, H*hd] of which the 2*len(inv_freq) elements of each head from `start` on are turned: as
    complex numbers (first, second element of pair i) times amplitude * exp(+-i pos inv_freq[i]), minus
    backward (the transposed map).  Half layout, or interleaved pairs; the rest is copied.  The angle's
    turns are reduced in exact rational arithmetic, so that it is right at every position."""
    from fractions import Fraction

    x = _f64(x)
    n, hd, d = x.shape[0], x.shape[1] // H, 2 * len(inv_freq)
    # 1 / (2 pi) to 2^-200, by Machin's formula for pi in integers
    one = 1 << 240
    arctan = lambda k: sum((1 if i % 2 == 0 else -1) * (one // k ** (2 * i + 1) // (2 * i + 1)) for i in range(120))
    turn = Fraction(one, 2 * 4 * (4 * arctan(5) - arctan(239)))
    ang = np.empty((n, d // 2))
    for i, f in enumerate(inv_freq):
        per = Fraction(float(f)) * turn
        per = Fraction(round(per * 2 ** 150), 2 ** 150)
        for r in range(n):
            t = int(pos[r]) * per
            ang[r, i] = float(t - round(t)) * 2 * np.pi
    z = amplitude * np.exp((-1j if backward else 1j) * ang)[:, None, :]
    out = x.reshape(n, H, hd).copy()
    part = out[:, :, start:start + d]
    if interleaved:
        w = (part[:, :, 0::2] + 1j * part[:, :, 1::2]) * z
        part[:, :, 0::2], part[:, :, 1::2] = w.real, w.imag
    else:
        w = (part[:, :, :d // 2] + 1j * part[:, :, d // 2:]) * z
        part[:, :, :d // 2], part[:, :, d // 2:] = w.real, w.imag
    return out.reshape(x.shape)


# ------------------------------------------------------------ paged key/value cache
F8_TOP = {"e4m3": 448.0, "e5m2": 57344.0}


def f8_values(kind):
    """The 256 values of an 8-bit floating type by code, from the type's definition:
    sign, exponent (4 bits, bias 7 | 5 bits, bias 15), fraction (3 | 2 bits), subnormals at
    exponent 0.  e4m3 has no infinity and NaN at 0x7f, 0xff; e5m2 is as IEEE."""
    eb, fb, bias = (4, 3, 7) if kind == "e4m3" else (5, 2, 15)
    out = np.zeros(256)
    for c in range(256):
        e, f = (c >> fb) & ((1 << eb) - 1), c & ((1 << fb) - 1)
        x = (f / (1 << fb)) * 2.0 ** (1 - bias) if e == 0 else (1 + f / (1 << fb)) * 2.0 ** (e - bias)
        if kind == "e4m3" and (c & 0x7f) == 0x7f:
            x = np.nan
        if kind == "e5m2" and e == 31:
            x = np.inf if f == 0 else np.nan
        out[c] = -x if c & 0x80 else x
    return out


def f8_round(x, kind):
    """Codes of the nearest values, ties to the even code; beyond the largest finite value
    (infinities too), the largest; NaN to the code 0x7f."""
    x = np.asarray(x, np.float64)
    top = {"e4m3": 0x7e, "e5m2": 0x7b}[kind]
    pos = f8_values(kind)[:top + 1]  # the finite values from 0 up: codes 0 .. top
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), pos[-1])
    hi = np.clip(np.searchsorted(pos, a), 1, top)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(x), 0x7f, code)
    return (code + 0x80 * np.signbit(x)).astype(np.uint8)


def turn_rows(x, pos, hd, theta):
    """Rows x [n, heads*hd] with the head vectors of row i turned as rope() does at
    position pos[i] (all rows at once)."""
    x = _f64(x)
    n = x.shape[0]
    y = x.reshape(n, x.shape[1] // hd, 2, hd // 2)
    ang = np.asarray(pos, np.float64)[:, None] * float(theta) ** (-2.0 * np.arange(hd // 2) / hd)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    return np.stack([y[:, :, 0] * c - y[:, :, 1] * s, y[:, :, 1] * c + y[:, :, 0] * s], 2).reshape(x.shape)


def paged_tokens(cache, scale, pages, n, kind=None):
    """Tokens 0 .. n-1 of one sequence as rows [n, Hkv*hd]: token t is row t % page of page
    pages[t // page] of cache [num_pages, Hkv, page, hd] (values, or codes of `kind` times
    the scale of their page and head); rows of a page outside the pool are NaN."""
    P, Hkv, page, hd = cache.shape
    out = np.full((n, Hkv, hd), np.nan)
    for t in range(n):
        pg = int(pages[t // page])
        if 0 <= pg < P:
            x = cache[pg, :, t % page]
            out[t] = x if kind is None else f8_values(kind)[x] * np.asarray(scale, np.float64)[pg][:, None]
    return out.reshape(n, Hkv * hd)


def paged_append(k, v, k_cache, v_cache, k_scale, v_scale, table, lengths, cu, *, Hkv, kind=None, theta=None):
    """What an append leaves: (k_cache, v_cache, k_scale, v_scale, exact) as new arrays.
    Rows cu[b] .. cu[b+1]-1 of k, v are sequence b's tokens at positions lengths[b] - n_b ..
    lengths[b] - 1; rows at a negative position, past the table or in a page outside the
    pool are dropped.  For 8-bit caches the block rule of the header, and `exact` lists
    (which, page, row, unrounded values [Hkv, hd] in units of the scale) of every new row."""
    P, _, page, hd = k_cache.shape
    out = [np.array(k_cache), np.array(v_cache)]
    sc = [None if s is None else np.array(s, np.float64) for s in (k_scale, v_scale)]
    exact = []
    for b in range(len(lengths)):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        first = int(lengths[b]) - (r1 - r0)
        pos = np.arange(first, int(lengths[b]))
        rows = [turn_rows(k[r0:r1], pos, hd, theta) if theta else _f64(k[r0:r1]), _f64(v[r0:r1])]
        for j in sorted({int(p) // page for p in pos if p >= 0}):
            if j >= table.shape[1] or not 0 <= int(table[b, j]) < P:
                continue
            pg = int(table[b, j])
            lo, hi = max(first, j * page, 0), min(int(lengths[b]), (j + 1) * page)
            for w in range(2):
                x = rows[w][lo - first:hi - first].reshape(hi - lo, Hkv, hd).transpose(1, 0, 2)
                at = lo - j * page
                if kind is None:
                    out[w][pg, :, at:at + hi - lo] = x
                    continue
                for h in range(Hkv):
                    mag = np.abs(x[h])
                    mag = mag[np.isfinite(mag)].max(initial=0.0)
                    s = 2.0 ** -64
                    while F8_TOP[kind] * s < mag:
                        s *= 2.0
                    if at > 0:
                        old = sc[w][pg, h]
                        if abs(old) >= s:
                            s = old
                        else:
                            out[w][pg, h, :at] = f8_round(f8_values(kind)[out[w][pg, h, :at]] * (old / s), kind)
                    sc[w][pg, h] = s
                    out[w][pg, h, at:at + hi - lo] = f8_round(x[h] / s, kind)
                for i in range(hi - lo):
                    exact.append((w, pg, at + i, x[:, i] / sc[w][pg][:, None]))
    return out[0], out[1], sc[0], sc[1], exact


def paged_decode(q, tokens, lengths, *, H, Hkv, scale, causal=True, window=0, softcap=0.0, absolute=False):
    """O [B, Lq, H*hd] and LSE [B, H, Lq] of Lq rows at positions lengths[b] - Lq ..
    lengths[b] - 1 over tokens[b] = (k, v), rows [lengths[b], Hkv*hd] (rows of NaN keys are
    not visible).  With `absolute`, V enters by its magnitude."""
    q = _f64(q)
    B, Lq, C = q.shape
    hd = C // H
    o, lse = np.zeros_like(q), np.full((B, H, Lq), -np.inf)
    for b in range(B):
        n = int(lengths[b])
        k, v = tokens[b]
        for i in range(Lq):
            p = n - Lq + i
            j = np.arange(n)
            j = j[~np.isnan(k[:, 0])] if n else j
            if causal:
                j = j[j <= p]
            if window:
                j = j[np.abs(p - j) < window]
            if j.size == 0:
                continue
            kk, vv = k[j].reshape(-1, Hkv, hd), v[j].reshape(-1, Hkv, hd)
            vv = np.abs(vv) if absolute else vv
            for h in range(H):
                s = scale * (kk[:, h // (H // Hkv)] @ q[b, i, h * hd:(h + 1) * hd])
                s = softcap * np.tanh(s / softcap) if softcap > 0 else s
                m = s.max()
                e = np.exp(s - m)
                o[b, i, h * hd:(h + 1) * hd] = e @ vv[:, h // (H // Hkv)] / e.sum()
                lse[b, h, i] = m + np.log(e.sum())
    return o, lse


def paged_prefill(q, tokens, lengths, cu, *, H, Hkv, scale, causal=True, window=0, softcap=0.0, absolute=False):
    """O [rows, H*hd] and LSE [H, rows] of packed rows: rows cu[b] .. cu[b+1]-1 are sequence b's last tokens,
    at positions lengths[b] - n_b .. lengths[b] - 1 over tokens[b] = (k, v), rows [lengths[b], Hkv*hd] (rows of
    NaN keys are not visible).  Rows in no sequence are NaN.  With `absolute`, V enters by its magnitude."""
    q = _f64(q)
    hd = q.shape[1] // H
    o, lse = np.full_like(q, np.nan), np.full((H, q.shape[0]), np.nan)
    for b in range(len(lengths)):
        r0, r1, n = int(cu[b]), int(cu[b + 1]), int(lengths[b])
        k, v = (np.asarray(x, np.float64).reshape(n, Hkv, hd) for x in tokens[b])
        p, j = (n - (r1 - r0) + np.arange(r1 - r0))[:, None], np.arange(n)[None, :]
        seen = np.broadcast_to(~np.isnan(k[:, 0, 0])[None, :], (r1 - r0, n))
        if causal:
            seen = seen & (j <= p)
        if window:
            seen = seen & (np.abs(p - j) < window)
        # (what no row sees may be anything)
        k = np.where(seen.any(0)[:, None, None], k, 0.0) if n else k
        v = np.where(seen.any(0)[:, None, None], v, 0.0) if n else v
        v = np.abs(v) if absolute else v
        for h in range(H):
            c = slice(h * hd, (h + 1) * hd)
            s = scale * (q[r0:r1, c] @ k[:, h // (H // Hkv)].T)
            s = softcap * np.tanh(s / softcap) if softcap > 0 else s
            s = np.where(seen, s, -np.inf)
            m = s.max(axis=1, initial=-np.inf)
            e = np.exp(s - np.where(np.isneginf(m), 0.0, m)[:, None])
            l = e.sum(1)
            o[r0:r1, c] = np.where(l[:, None] > 0, e @ v[:, h // (H // Hkv)] / np.where(l > 0, l, 1.0)[:, None], 0.0)
            with np.errstate(divide="ignore"):
                lse[h, r0:r1] = np.where(l > 0, m + np.log(l), -np.inf)
    return o, lse

"""Host-side refusals of the paged-chunk attention, the rotating append and the
norm with rotation (CPU; nothing is launched)."""
import ctypes
import math

import pytest

from exact_attention_41_gb300 import build as build_mod
from exact_attention_41_gb300 import libattn

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)
BYTE = ctypes.c_void_p(0x10002)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return libattn.lib()


def paged(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE, q_rs=0, k_ps=0, v_ps=0, cu=FAKE, cs=FAKE,
             bt=FAKE, num_pages=8, page=64, max_pages=4, appended=1, batch=2, total=8, dtype=1, hq=4,
             hkv=2, d=128, scale=0.1, causal=1, wl=-1, wr=-1, cap=0.0, splits=0, ws=FAKE, n=BIG)
    a.update(over)
    return lib.attn_fwd_paged(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(d=96), 2), (dict(hq=5), 1), (dict(dtype=2), 1), (dict(batch=-1), 1), (dict(total=-1), 1),
    (dict(page=0), 1), (dict(page=-16), 1), (dict(max_pages=0), 1), (dict(num_pages=-1), 1),
    (dict(splits=-1), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(out=None), 1),
    (dict(lse=None), 1), (dict(cu=None), 1), (dict(cs=None), 1), (dict(q=ODD), 1), (dict(v=ODD), 1),
    (dict(lse=BYTE), 1), (dict(cu=BYTE), 1), (dict(cs=BYTE), 1), (dict(bt=BYTE), 1),
    (dict(q_rs=4 * 128 - 8), 1), (dict(q_rs=4 * 128 + 4), 1), (dict(k_ps=64 * 2 * 128 - 8), 1),
    (dict(v_ps=64 * 2 * 128 + 4), 1), (dict(bt=None), 1), (dict(bt=None, num_pages=2), 1),
    (dict(scale=float("nan")), 1), (dict(wl=-2), 1), (dict(cap=float("nan")), 1),
    (dict(max_pages=1 << 26), 2), (dict(splits=8, n=0), 3), (dict(splits=8, ws=None), 3),
    (dict(batch=0), 0), (dict(total=0), 0),
])
def test_paged_refusals(lib, over, status):
    assert paged(lib, **over) == status


def test_paged_workspace_size(lib):
    size = lib.attn_fwd_paged_workspace_size
    assert size(4, 100, 32, 8, 128, 1) == 0          # one key range per row: no partials
    assert size(0, 100, 32, 8, 128, 0) == 0 and size(4, 0, 32, 8, 128, 0) == 0
    # 4 key ranges: at least the partial outputs of every row
    assert size(4, 100, 32, 8, 128, 4) >= 4 * 100 * 32 * 129 * 4
    assert size(1, 1, 8, 8, 64, 0) > 0


def rope(lib, **over):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, s0=0, s1=0, s2=0, s3=0, wq=FAKE, wk=FAKE, eps=1e-6,
             ph=FAKE, rot=128, inter=0, pos=None, dtype=1, b=1, s=8, hq=4, hkv=2, d=128)
    a.update(over)
    return lib.attn_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(d=80), 2), (dict(dtype=-1), 1), (dict(rot=8), 1), (dict(rot=144), 1), (dict(rot=-16), 1),
    (dict(ph=None), 1), (dict(ph=ODD), 1), (dict(pos=BYTE), 1), (dict(wq=ODD), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("inf")), 1), (dict(q=None), 1), (dict(ko=None), 1), (dict(qo=ODD), 1),
    (dict(s0=4 * 128 - 8), 1), (dict(s2=4 * 128 + 1), 1), (dict(b=-1), 1), (dict(hq=-1), 1),
    (dict(s2=4 * 128 + 8), 1),                       # in place (q_out is q), other row places
    (dict(b=1 << 15, s=1 << 15), 2), (dict(b=0), 0), (dict(s=0), 0), (dict(hq=0, hkv=0), 0),
])
def test_norm_rope_refusals(lib, over, status):
    assert rope(lib, **over) == status


def test_norm_rope_backward_refusals(lib):
    def call(**over):
        a = dict(q=FAKE, k=FAKE, gq=FAKE, gk=FAKE, dq=FAKE, dk=FAKE, s0=0, s1=0, s2=0, s3=0,
                 wq=FAKE, wk=FAKE, dwq=FAKE, dwk=FAKE, eps=1e-6, ph=FAKE, rot=64, inter=0, pos=None,
                 dtype=0, b=2, s=8, hq=4, hkv=2, d=64, ws=FAKE, n=BIG)
        a.update(over)
        return lib.attn_qk_norm_rope_bwd(*a.values(), None)

    assert call(dwq=None) == 1 and call(dk=None) == 1 and call(q=None) == 1
    assert call(n=16) == 3 and call(ws=None) == 3
    assert call(ws=ODD) == 1 and call(rot=72) == 1 and call(d=32) == 2 and call(pos=BYTE) == 1
    assert call(s2=4 * 64 + 8) == 1                  # dq is dq_out, but in other row places
    assert call(hq=0, hkv=0) == 0
    assert lib.attn_qk_norm_rope_bwd_workspace_size(0, 8, 4, 2, 64) == 0


def test_append_refusals(lib):
    def call(**over):
        a = dict(q=FAKE, qo=FAKE, k=FAKE, v=FAKE, s0=0, s1=0, s2=0, kc=FAKE, vc=FAKE, kp=0, vp=0,
                 cu=FAKE, cs=FAKE, bt=FAKE, num_pages=8, page=5, max_pages=4, wq=None, wk=None,
                 eps=0.0, ph=FAKE, rot=64, inter=1, dtype=1, batch=2, total=8, hq=4, hkv=2, d=64)
        a.update(over)
        return lib.attn_kvcache_append(*a.values(), None)

    for over in (dict(k=None), dict(v=None), dict(qo=None), dict(kc=None), dict(cu=None),
                 dict(cs=None), dict(page=0), dict(kp=5 * 2 * 64 - 8), dict(vp=5 * 2 * 64 + 4),
                 dict(hkv=0), dict(rot=24), dict(s1=8), dict(bt=None), dict(vc=ODD),
                 dict(cu=BYTE), dict(cs=BYTE), dict(bt=BYTE), dict(total=-1), dict(batch=-1)):
        assert call(**over) == 1, over
    assert call(total=0) == 0 and call(batch=0) == 0


def test_phases(lib):
    """Fractions of a turn per position in units of 2^-64 turns."""
    turn = 2 * math.pi
    phase = lib.attn_rope_phase
    assert phase(0.0) == 0
    for f in (1.0, 0.1, 1e-5, 3.0, turn / 4):
        want = f / turn
        assert abs(phase(f) / 2.0 ** 64 - (want - math.floor(want))) < 2 ** -52
    # a frequency and its negative cancel; whole turns do not count
    assert (phase(0.7) + phase(-0.7)) % 2 ** 64 < 2 ** 13 or \
        2 ** 64 - (phase(0.7) + phase(-0.7)) % 2 ** 64 < 2 ** 13
    # far positions keep the angle: compare with exact rational arithmetic
    from fractions import Fraction

    f, pos = 0.31622776601683794, 10 ** 9
    exact = Fraction(f) / (2 * Fraction("3.14159265358979323846264338327950288")) * pos
    frac = float(exact - math.floor(exact))
    got = (phase(f) * pos % 2 ** 64) / 2.0 ** 64
    assert abs(got - frac) < 1e-6   # the 64-bit frequency itself: 2^-53 * 0.05 * 1e9 = 6e-9 turns


def test_phases_of_what_is_no_frequency(lib):
    for f in (float("inf"), float("-inf"), float("nan")):
        assert lib.attn_rope_phase(f) == 0
    assert lib.attn_rope_phases(FAKE, FAKE, -1, None) == 1
    assert lib.attn_rope_phases(None, FAKE, 4, None) == 1
    assert lib.attn_rope_phases(FAKE, ctypes.c_void_p(0x10004), 4, None) == 1
    assert lib.attn_rope_phases(None, None, 0, None) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        libattn.qk_norm_rope(q, q)
    with pytest.raises(ValueError, match="share"):
        libattn.qk_norm_rope(q, q.half())
    with pytest.raises(ValueError, match="needed"):
        libattn.qk_norm_rope(None, None)
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    cu, cs = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="int32"):
        libattn.fwd_paged(q[0], pool, pool, cu.long(), cs)
    with pytest.raises(ValueError, match="one entry more"):
        libattn.fwd_paged(q[0], pool, pool, cu[:2], cs)
    with pytest.raises(ValueError, match="CUDA"):
        libattn.fwd_paged(q[0], pool, pool, cu, cs)
    with pytest.raises(ValueError, match="CUDA"):
        libattn.kvcache_append(q[0], q[0], pool, pool, cu, cs)


def test_expanded_tensors_are_refused():
    """A stride of 0 stands for contiguous rows in the C calls: an expanded
    tensor, which has it, would be read past its end."""
    torch = pytest.importorskip("torch")
    row = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expanded"):
        libattn._packed_stride(row.expand(4, 2, 64))
    assert libattn._packed_stride(row) == 0
    page = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expanded"):
        libattn._page_stride(page.expand(4, 16, 2, 64))
    assert libattn._page_stride(page) == 0
    wide = torch.zeros(4, 3, 2, 64, dtype=torch.bfloat16)
    assert libattn._packed_stride(wide[:, 0]) == 3 * 2 * 64

    class OnDevice:  # the layout of a CUDA tensor, without one
        is_cuda, shape = True, (1, 4, 2, 64)

        def is_contiguous(self):
            return False

        def stride(self, i):
            return (0, 0, 64, 1)[i]

    with pytest.raises(ValueError, match="expanded"):
        libattn._row_stride(OnDevice())


def test_numbers_beyond_a_c_int():
    import sys

    for x, want in ((2 ** 32, 2 ** 31 - 1), (sys.maxsize, 2 ** 31 - 1), (-2 ** 40, -2 ** 31), (-1, -1),
                    (2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, -2 ** 31)):
        assert libattn._int(x) == want

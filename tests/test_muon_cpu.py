"""The matrix optimizer's argument checks, which come before any device call."""
from __future__ import annotations

import ctypes as C

import pytest
import torch

import zero_sharded_adamw_gb300 as z
from tests.test_abi_cpu import CTYPES, _struct_fields
from zero_sharded_adamw_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


@pytest.mark.parametrize("struct,binding", [("zero1_matrix", z._CMatrix), ("zero1_muon_hparams", z._CMuonHparams)])
def test_structs_match_header(struct, binding):
    fields = _struct_fields(struct)
    assert [n for n, _ in fields] == [n for n, _ in binding._fields_]
    for (_, ctype), (_, bt) in zip(fields, binding._fields_):
        assert CTYPES[ctype] is bt


def refused(*args, **kw):
    with pytest.raises(z.Zero1Error) as e:
        z.zero1_muon_create(*args, **kw)
    return e.value.code, str(e.value)


def accepted(n, mats):
    """Passes every check: only the device is missing here (or it is there)."""
    try:
        z.zero1_muon_destroy(z.zero1_muon_create(n, 1, mats))
    except z.Zero1Error as e:
        assert e.code == -5, e


@pytest.mark.parametrize("hp", [dict(lr=-1.0), dict(lr=float("nan")), dict(momentum=1.0), dict(momentum=-0.1),
                                dict(weight_decay=float("inf")), dict(eps=0.0), dict(eps=1e-16), dict(update_scale=-1.0),
                                dict(nesterov=2), dict(scale_rule=5), dict(ns_steps=0), dict(ns_steps=33),
                                dict(ns_a=float("nan")), dict(ns_b=9.0), dict(ns_c=0.0), dict(ns_b=-4.0, ns_c=0.4), dict(inject_wait_timeout=2)])
def test_hyperparameters(hp):
    assert refused(64, 1, [(0, 8, 8)], z.MuonHparams(**hp))[0] == -1


@pytest.mark.parametrize("n,world,mats", [
    (0, 1, [(0, 1, 1)]), (64, 0, [(0, 8, 8)]), (64, z.ZERO1_MAX_WORLD + 1, [(0, 8, 8)]), (64, 1, []),
    (64, 1, [(0, 0, 8)]), (64, 1, [(0, 8, 0)]), (64, 1, [(0, 8, 8, 7)]), (63, 1, [(0, 8, 8)]), (64, 1, [(1, 8, 8)]),
    (64, 1, [(65, 1, 1)]), (1 << 60, 1, [(0, 8, 8)]), (64, 1, [(2**62, 8, 8)]), (64, 1, [(0, 1, (1 << 22) + 1)]),
    (1 << 40, 1, [(0, 8, 8, 2**62)]),
])
def test_sizes(n, world, mats):
    assert refused(n, world, mats)[0] == -1


def test_struct_size_is_checked():
    hp = z.MuonHparams()._c()
    hp.size = 8
    h = C.c_void_p()
    mats = (z._CMatrix * 1)(z._CMatrix(0, 8, 8, 8))
    assert z._load().zero1_muon_create(64, 1, mats, 1, C.byref(hp), C.byref(h)) == -1 and not h.value
    assert z._load().zero1_muon_create(64, 1, None, 1, C.byref(hp), C.byref(h)) == -1
    assert z._load().zero1_muon_create(64, 1, mats, 1, None, C.byref(h)) == -1
    assert z._load().zero1_muon_create(64, 1, mats, 1, C.byref(hp), None) == -1


@pytest.mark.parametrize("mats", [[(0, 8, 8), (63, 2, 2)], [(0, 8, 8), (0, 8, 8)], [(10, 4, 4, 16), (13, 4, 4, 16)],
                                  [(10, 4, 4, 16), (28, 1, 4, 16)], [(0, 4, 4, 16), (8, 2, 2, 20)],
                                  [(12, 4, 4, 16), (28, 4, 4, 16)], [(0, 4, 2, 8), (6, 4, 3, 8)]])
def test_overlaps(mats):
    code, msg = refused(1000, 1, mats)
    assert code == -1 and "overlap" in msg


def brute_force_overlap(mats):
    seen = set()
    for off, r, c, ld in mats:
        for i in range(r):
            for j in range(c):
                e = off + i * ld + j
                if e in seen:
                    return True
                seen.add(e)
    return False


def test_overlap_rule_against_enumeration():
    """Every pair of small matrices of one stride: refused exactly when they
    share an entry."""
    ld = 6
    for c1 in (1, 3, 6):
        for r1 in (1, 3):
            for c2 in (1, 2, 5):
                for r2 in (1, 2):
                    for off in range(0, 30):
                        mats = [(0, r1, c1, ld), (off, r2, c2, ld)]
                        if brute_force_overlap(mats):
                            assert refused(1000, 1, mats)[0] == -1, mats
                        else:
                            accepted(1000, mats)


def test_slices_and_any_order_are_taken():
    accepted(50 * 288, [(192, 50, 96, 288), (0, 50, 96, 288), (96, 50, 96, 288)])
    accepted(200, [(100, 10, 10), (0, 10, 10)])
    accepted(10, [(9, 1, 1), (0, 9, 1)])


def test_binding_checks():
    for mats in ([(0, 8)], [(0, 8, 8, 8, 8)], [(-1, 8, 8)], [(0, 1 << 33, 8)], [(1 << 63, 8, 8)]):
        with pytest.raises(z.Zero1ArgumentError):
            z.zero1_muon_create(64, 1, mats)
    with pytest.raises(z.Zero1ArgumentError):
        z._dtype_of(torch.zeros(4, dtype=torch.float16), "x")
    bogus = 0xDEAD0000
    for call in (lambda: z.zero1_muon_step(bogus, [16], [16], 16, 16), lambda: z.zero1_muon_set_lr(bogus, 1e-3),
                 lambda: z.zero1_muon_orthogonalize(bogus, 16, 0, 16, 0), lambda: z.zero1_muon_status(bogus),
                 lambda: z.zero1_muon_layout(bogus), lambda: z.zero1_muon_destroy(bogus)):
        with pytest.raises(z.Zero1Error) as e:
            call()
        assert e.value.code == -1
    z.zero1_muon_destroy(None)

"""Model check of the long-prefix kernel's synchronisation protocol
(csrc/paged_prefix.cu) on the CPU; see tests/prefix_protocol_model.py."""

import dataclasses
import os
import random
import re

import pytest

import prefix_protocol_model as PM

FORMS = {64: (2, 4, 4), 128: (2, 2, 3), 256: (1, 2, 3)}  # head_dim: lanes, K stages, V stages


@pytest.mark.parametrize("d", FORMS)
def test_random_pieces_and_schedules(d):
    for seed in range(250):
        rng = random.Random(seed)
        PM.PrefixModel(PM.random_pieces(rng, FORMS[d][0]), *FORMS[d], rng=rng, rescale_prob=rng.random()).run()


@pytest.mark.parametrize("d", FORMS)
@pytest.mark.parametrize("count", [1, 2, 3, 12])
def test_edge_tile_counts(d, count):
    lanes = FORMS[d][0]
    for seed in range(20):
        for apart in (False, True)[:lanes]:
            for p in (0.0, 1.0):
                piece = PM.Piece(count, apart, ((0, 1, 2, 3), (0,))[:lanes], seed % 2 == 0)
                if apart:
                    piece = dataclasses.replace(piece, valid=((0, 1), (0, 1)))
                PM.PrefixModel([piece] * (1 + seed % 3), *FORMS[d], rng=random.Random(seed), rescale_prob=p).run()


@pytest.mark.parametrize("slip", [f.name for f in dataclasses.fields(PM.PrefixMutation)])
def test_planted_protocol_slips_are_caught(slip):
    mut = PM.PrefixMutation(**{slip: True})
    for seed in range(600):
        rng = random.Random(seed)
        d = 256 if slip in ("one_place_barriers", "rescale_without_wait") else 128
        try:
            PM.PrefixModel(PM.random_pieces(rng, FORMS[d][0]), *FORMS[d], mut=mut, rng=rng, rescale_prob=0.5).run()
        except PM.ProtocolViolation:
            return
    pytest.fail("slip %s not caught in 600 schedules" % slip)


def test_model_matches_the_kernel_source():
    src = open(os.path.join(os.path.dirname(__file__), "..", "dynamic_hierarchical_sparse_b200", "csrc",
                            "paged_prefix.cu")).read()
    counts = dict(re.findall(r"mbar_init\(bar\((kBar\w+)(?: \+ \w+)?\), ([^;]+)\);", src))
    for name in ("kBarKFull", "kBarVFull", "kBarSFull", "kBarODone", "kBarTurn"):
        assert counts[name] == "1", name
    for name in ("kBarKFree", "kBarVFree"):
        assert counts[name] == "C::kLanes", name
    for name in ("kBarPHalf", "kBarPFull", "kBarQFull", "kBarCross"):
        assert counts[name] == "4", name
    assert counts["kBarPiece"] == "4 * C::kLanes"
    assert "kKStages = D == 64 ? 4 : 2;" in src and "kVStages = D == 64 ? 4 : 3;" in src
    assert "kLanes = D == 256 ? 1 : 2;" in src
    assert "return C::kLanes == 2 ? a : n & 1;" in src
    assert "(C::kLanes == 2 ? n : n >> 1) & 1" in src
    # one lane: S of the next tile, its K released, then P V; two: the turn holds P V, then S
    two, one = src[src.index("if constexpr (C::kLanes == 2) {\n              if (pv"):].split("} else {", 1)
    assert two.index("p_there()") < two.index("k_there()") < two.index("wait_turn") < two.index("send_pv()") < two.index("send_s()")
    assert one.index("send_s()") < one.index("kBarKFree") < one.index("p_there()") < one.index("send_pv()")

"""Every routing kernel that is compiled serves some router (CPU only: the
choice of shapes is worked out here for every router the library accepts, from
the shapes that the source names)."""
from __future__ import annotations

import os
import re

from copy_reduce_snac_amd.build import CSRC

MORE_ROUNDS = 3


def fits(experts, groups, topk, lanes, per_lane, most):
    shift = 0
    while per_lane << shift < experts // groups:
        shift += 1
    return topk <= most and topk + MORE_ROUNDS + 1 <= lanes and groups << shift <= lanes


def test_every_shape_is_reached():
    src = open(os.path.join(CSRC, "route.hip")).read()
    assert f"kMoreRounds = {MORE_ROUNDS};" in src
    body = src[src.index("void route_any("):]
    body = body[:body.index("\n}\n")]
    shapes = [tuple(map(int, m)) for m in re.findall(r"route_fits<T, (\d+), (\d+), (\d+), KEY>", body)]
    many, few = [s for s in shapes if s[0] < 64], [s for s in shapes if s[0] == 64]
    assert shapes == many + few and len(shapes) == 14  # those of many tokens are tried first
    reached, exact = set(), set()
    for experts in range(1, 1025):
        for groups in (g for g in range(1, 65) if experts % g == 0):
            for topk in range(1, min(32, experts) + 1):
                for tries in (shapes, few):
                    first = next((s for s in tries if fits(experts, groups, topk, *s)), None)
                    (reached.add(first) if first else exact.add(experts))
    assert reached == set(shapes)
    assert min(exact) == 561
    # so the kernel that works in binary64 throughout is needed at 16 experts a lane only
    assert set(re.findall(r"route_exact_kernel<T, (\d+)>", src)) == {"16"}

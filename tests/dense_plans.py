"""The plans of the dense block's products, read from the kernel's source: the
instance tables, and the choice of an instance and of the shares of a sum
(f32 arithmetic, as the library's)."""

import os
import re

import numpy as np

from moe_grouped_gemm_route_amd import build

F32 = np.float32


def _source():
    with open(os.path.join(build.CSRC, "gateup.hip")) as f:
        return f.read()


def tables():
    """{name: [(rows, columns, groups, fit, stage, alone)]} of the TileConfig tables."""
    out = {}
    for name, body in re.findall(r"static const TileConfig (k\w+)\[\] = \{(.*?)\};", _source(), re.S):
        rows = re.findall(r"\{(\d+), (\d+), (\d+), (\d+), ([\d.]+)f, ([\d.]+)f\}", body)
        out[name] = [tuple(map(int, r[:4])) + (F32(r[4]), F32(r[5])) for r in rows]
    return out


def constant(name):
    return int(re.search(r"constexpr int %s = (\d+);" % name, _source()).group(1))


class Plans:
    def __init__(self):
        self.tables = tables()
        self.bk, self.cus, self.most = constant("GU_BK"), constant("GU_CUS"), constant("GU_SPLITS")

    def plan(self, table, rows, cols, depth):
        """(instance, shares) for out [rows, cols], a sum over depth (kForward:
        columns of h, no shares)."""
        gate = table == "kForward"
        best, least = (0, 1), F32(0)
        for c, (bm, bn, kg, fit, stage, alone) in enumerate(self.tables[table]):
            tiles = -(-rows // bm) * -(-cols // (bn // 2 if gate else bn))
            stages = -(-(-(-depth // self.bk)) // kg)
            shares = 1
            while shares <= (1 if gate else self.most) and shares <= stages:
                if shares > 1 and tiles * shares > 2 * fit:
                    break
                one = alone if tiles * shares <= self.cus else stage
                us = F32(-(-tiles * shares // fit)) * (F32(3) + F32(-(-stages // shares) * kg) * one)
                if shares > 1:
                    us = us + (F32(4) + F32(shares) * F32(rows) * F32(cols) * F32(F32(8) / F32(4.5e6)))
                if least == 0 or us < least:
                    best, least = (c, shares), us
                shares *= 2
        return best

    def of(self, M, N, K):
        """Every plan that calls of these sizes take, {(table, instance, shares)}."""
        out = {("kForward",) + self.plan("kForward", M, N // 2, K)} if M > 16 else set()
        for table in ("kDx", "kDx3"):
            out.add((table,) + self.plan(table, M, K, N))
        for table in ("kDw", "kDw3"):
            out.add((table,) + self.plan(table, N, K, M))
        return out

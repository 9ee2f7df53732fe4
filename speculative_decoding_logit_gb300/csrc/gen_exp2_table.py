"""Build step: write exp2_table.inc, the table of the sampling's accurate weights.

Entry j of 64 is 2^(j/64) as an unevaluated sum of two floats: the value rounded to fp32, and what that
leaves, rounded to fp32 again (2^-49 of the value are lost).  The scheme is Tang's table-driven exponential
(P. T. P. Tang, "Table-driven implementation of the exponential function in IEEE floating-point arithmetic",
ACM TOMS 15 (1989)): 2^t = 2^e 2^(j/64) 2^r with |r| <= 2^-7.

Run:  python gen_exp2_table.py   (rewrites exp2_table.inc beside this file)
"""
import os

import mpmath as mp
import numpy as np

mp.mp.dps = 50


def split(v):
    hi = np.float32(float(v))
    return float(hi), float(np.float32(float(v - mp.mpf(float(hi)))))


def main():
    lines = ["// Generated by gen_exp2_table.py -- do not edit.",
             "// 2^(j/64) = hi + lo, and ln 2 = hi + lo.",
             "static __device__ const float2 kExp2Table[64] = {"]
    for j in range(64):
        hi, lo = split(mp.mpf(2) ** (mp.mpf(j) / 64))
        lines.append(f"    {{{hi.hex()}f, {lo.hex()}f}},")
    hi, lo = split(mp.log(2))
    lines += ["};", f"constexpr float kLn2Hi = {hi.hex()}f, kLn2Lo = {lo.hex()}f;"]
    hi, lo = split(1 / mp.log(2))
    lines += [f"constexpr float kLog2eHi = {hi.hex()}f, kLog2eLo = {lo.hex()}f;"]
    with open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "exp2_table.inc"), "w") as f:
        f.write("\n".join(lines) + "\n")


if __name__ == "__main__":
    main()

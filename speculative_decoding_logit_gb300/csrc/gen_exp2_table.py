"""Build step: write exp2_table.inc, the table of the sampling's exact weights.

Entry j of 1024 is 2^(j/1024) in units of 2^-30, rounded.  The scheme is Tang's table-driven exponential
(P. T. P. Tang, "Table-driven implementation of the exponential function in IEEE floating-point arithmetic",
ACM TOMS 15 (1989)): 2^t = 2^e 2^(j/1024) 2^r with |r| <= 2^-11.  ln 2 and log2 e as unevaluated sums of two
floats: the value rounded to fp32, and what that leaves, rounded to fp32 again.

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
             "// 2^(j/1024) in units of 2^-30; ln 2 = hi; log2 e = hi + lo.",
             "static __device__ const uint32_t kExp2Table[1024] = {"]
    table = [int(mp.nint(mp.mpf(2) ** (mp.mpf(j) / 1024) * 2 ** 30)) for j in range(1024)]
    for j in range(0, 1024, 8):
        lines.append("    " + " ".join(f"0x{v:x}u," for v in table[j:j + 8]))
    hi, _ = split(mp.log(2))
    lines += ["};", f"constexpr float kLn2Hi = {hi.hex()}f;"]
    hi, lo = split(1 / mp.log(2))
    lines += [f"constexpr float kLog2eHi = {hi.hex()}f, kLog2eLo = {lo.hex()}f;"]
    with open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "exp2_table.inc"), "w") as f:
        f.write("\n".join(lines) + "\n")


if __name__ == "__main__":
    main()

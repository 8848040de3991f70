"""The cosine and sine of the rotary positions (cos_sin.h), built for the host: as near as their
comment says, which how often a rotated key's code can differ from the oracle's depends on.

Bound, relative to first order in u = 2^-53, for |x| <= 2^31: the series leave out less than r^17/17! and
r^18/18!, 0.6 u of the sine at |r| = pi/4; r is rounded once (u; x - n pi/2 with the first part of pi/2
is exact), which moves the cosine by r tan r u < 0.8 u; the last sum rounds once (u of the sine, 1.42 u
of the cosine, which is at least 0.707 and has numbers u/2 .. u apart), and the terms before it are
at most 0.15 and 0.44 of the values with three roundings each at most: below 4 u = 2^-51 in all.  Near
a zero of either the two parts of pi/2 count, 2^-109 off it together: 2^-78 at n = 2^31 2/pi."""

import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_weight_only_quantize_amd", "csrc")


def test_cosine_and_sine_are_as_good_as_they_say():
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "cos_sin")
        subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-I", CSRC,
                        os.path.join(HERE, "cos_sin_check.cpp"), "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, timeout=300, check=True).stdout
    for line in out.split("\n")[:2]:
        worst, at = (float(x) for x in line.split())
        assert worst <= 2.0 ** -51, (worst, at)

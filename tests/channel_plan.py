"""csrc/channel_plan.h for tests: compiled by the host compiler, with the room
that 152 SMs have, and the form that a product of given sizes takes."""
import ctypes
import functools
import os
import subprocess
import tempfile

from w4a16_linear_layers_gb300 import build as qbuild

# clusters that run at one time on 152 SMs, by their size from 1 on
PAIRS = (76, 36, 23, 15)
NARROW = (456, 228, 148, 110, 87, 74, 59, 51)
WIDE = (304, 152, 97, 74, 58, 46, 38, 36)
TOKENS16 = WIDE

SHIM = r"""
#include "channel_plan.h"
using namespace qlin;
static Room room() {
  Room r;
  r.sm_count = 152;
  const int pairs[] = {%s}, narrow[] = {%s}, wide[] = {%s}, tokens16[] = {%s};
  static_assert(sizeof(pairs) == kMaxParts * sizeof(int) && sizeof(narrow) == kMaxSplits * sizeof(int), "sizes");
  for (int i = 0; i < kMaxParts; ++i) r.pairs[i + 1] = pairs[i];
  for (int i = 0; i < kMaxSplits; ++i) {
    r.narrow[i + 1] = narrow[i];
    r.wide[i + 1] = wide[i];
    r.tokens16[i + 1] = tokens16[i];
  }
  return r;
}
extern "C" int plan_streams(int64_t M, int64_t N, int64_t K) { return streams(M, N, K, room()); }
extern "C" void plan_stream3(int64_t M, int64_t N, int64_t K, int64_t* o) {
  const StreamPlan p = plan_stream(M, N, K, room());
  o[0] = p.channels; o[1] = p.tokens; o[2] = p.splits;
}
extern "C" void plan_pair12(int64_t M, int64_t N, int64_t K, int64_t* o) {
  const PairPlan p = plan_pair(M, N, K, room());
  o[0] = p.T; o[1] = p.TT; o[2] = p.F2; o[3] = p.G; o[4] = p.pairs; o[5] = p.band; o[6] = p.sk_tiles;
  o[7] = p.sk_pairs; o[8] = p.parts; o[9] = p.cut; o[10] = (int64_t)p.part_bytes; o[11] = p.cost;
}
extern "C" int64_t plan_workspace(int64_t M, int64_t N, int64_t K, int c16) {
  return (int64_t)plan_workspace_bytes(M, N, K, c16 != 0, room());
}
"""
FIELDS = ("T", "TT", "F2", "G", "pairs", "band", "sk_tiles", "sk_pairs", "parts", "cut", "part_bytes", "cost")


@functools.lru_cache(None)
def lib():
    with tempfile.TemporaryDirectory() as d:
        src, out = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SHIM % tuple(", ".join(map(str, t)) for t in (PAIRS, NARROW, WIDE, TOKENS16)))
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC", "-shared", "-I", qbuild.CSRC, src,
                        "-o", out], check=True)
        so = ctypes.CDLL(out)
    I, P = ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)
    so.plan_streams.argtypes = [I, I, I]
    so.plan_stream3.argtypes = so.plan_pair12.argtypes = [I, I, I, P]
    so.plan_workspace.argtypes = [I, I, I, ctypes.c_int]
    so.plan_workspace.restype = I
    return so


def streams(M, N, K):
    return bool(lib().plan_streams(M, N, K))


def stream_plan(M, N, K):
    o = (ctypes.c_int64 * 3)()
    lib().plan_stream3(M, N, K, o)
    return tuple(o)


def pair_plan(M, N, K):
    o = (ctypes.c_int64 * 12)()
    lib().plan_pair12(M, N, K, o)
    return dict(zip(FIELDS, o))


def workspace_bytes(M, N, K, c16):
    return int(lib().plan_workspace(M, N, K, int(c16)))


def form(M, K, N):
    """("stream", channels, tokens, blocks of a cluster) or ("pair", T, how):
    "direct": whole tiles of one accumulator, "sums": whole tiles of several,
    "shared2" to "shared4": tiles shared in a cluster, "parts": the last tiles
    cut into equal parts, "across": into shares that cross tiles."""
    if streams(M, N, K):
        return ("stream", *stream_plan(M, N, K))
    p = pair_plan(M, N, K)
    if p["parts"] > 1:
        how = f"shared{p['parts']}"
    elif p["cut"]:
        how = "parts" if p["sk_pairs"] % p["sk_tiles"] == 0 else "across"
    else:
        how = "direct" if p["G"] <= 8 else "sums"
    return ("pair", p["T"], how)

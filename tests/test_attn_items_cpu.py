"""The lists of items that memq_attn_paged's kernels walk, compiled on the host: over lengths that stand still each
item comes once; over lengths that change between two reads nothing outside the arrays is named."""
import os
import re
import shutil
import subprocess

import pytest

from quantized_decode_memq_gb300.build import CSRC

PROGRAM = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>
#define __device__
#define __host__
#define __forceinline__ inline
using std::max;
using std::min;
static bool moving = false;  // every read of a length gives another number
static uint64_t state = 7;
static uint32_t next() { state = state * 6364136223846793005ull + 1442695040888963407ull; return state >> 33; }
static int32_t __ldcg(const int32_t *p) {
    if (!moving) return *p;
    switch (next() % 5) {
        case 0: return static_cast<int32_t>(next() << 1);
        case 1: return 0;
        default: return static_cast<int32_t>(next() % 40) - 2;
    }
}
struct AttnArgs {
    const int32_t *kv_len, *cu_q;
    int n_tok, n_seq, n_kv, group, max_pages, page_shift, rows_from, rows_to;
};
SOURCE

static long errors = 0;
static void inside(const AttnArgs &a, int seq, int head, const AttnSeq &s, int row0, int n_rows, int vis, const char *what) {
    const bool rows = n_rows > 0, keys = vis > 0;
    bool ok = head >= 0 && head < a.n_kv && row0 >= 0;
    if (rows) ok = ok && s.start >= 0 && s.start + (row0 + n_rows - 1) / a.group < a.n_tok;
    if (keys) ok = ok && seq >= 0 && seq < a.n_seq && vis <= (static_cast<long long>(a.max_pages) << a.page_shift);
    if (!ok && errors++ < 10) std::printf("%s: seq %d head %d row0 %d n_rows %d vis %d\n", what, seq, head, row0, n_rows, vis);
}

int main() {
    for (int i = 0; i < 4000; ++i) {
        AttnArgs a{};
        a.n_seq = 1 + next() % 6;
        a.n_kv = 1 + next() % 3;
        a.group = 1 + next() % 9;
        a.page_shift = 4;
        a.max_pages = 1 + next() % 8;
        a.rows_from = 1;
        a.rows_to = 0x7fffffff;
        std::vector<int32_t> cu(a.n_seq + 1, 0), kv(a.n_seq, 0);
        for (int b = 0; b < a.n_seq; ++b) {
            cu[b + 1] = cu[b] + (next() % 3 ? next() % 30 : 0);
            kv[b] = next() % (a.max_pages * 16 + 1);
        }
        a.n_tok = max(1, cu[a.n_seq]);
        a.cu_q = cu.data();
        a.kv_len = kv.data();
        int first = 0;
        while (first < a.n_seq && cu[first + 1] == cu[first]) ++first;
        if (first == a.n_seq) continue;
        const AttnSeq s0{cu[first], cu[first + 1] - cu[first], kv[first]};
        long want_rows = 0, want_tiles = 0;
        for (int b = 0; b < a.n_seq; ++b) {
            const int rows = (cu[b + 1] - cu[b]) * a.group;
            want_rows += static_cast<long>((rows + kRows - 1) / kRows) * a.n_kv;
            want_tiles += static_cast<long>((rows + 127) / 128) * a.n_kv;
        }
        for (int turn = 0; turn < 2; ++turn) {
            // the row kernel's items
            moving = false;
            RowItem it{};
            it.seq = first;
            it.s = s0;
            it.of_seq(a);
            const long long far = 1ll << 40;
            it.sizes(a, far);
            moving = turn == 1;
            long n = 0;
            for (; it.live && n < 3000; it.advance(a, far), ++n)
                inside(a, it.seq, it.head, it.s, it.row0, it.n_rows, it.vis, "rows");
            if (!moving && n != want_rows) ++errors, std::printf("rows: %ld items of %ld\n", n, want_rows);
            // the tensor-core kernel's, some way past the last
            moving = false;
            TileItem t{};
            if (turn == 0 || next() % 2) {  // or the item that stands there until a thread notes the first
                t.seq = first;
                t.s = s0;
                t.rows = s0.t * a.group;
                tile_sizes(a, 128, t);
            }
            moving = turn == 1;
            for (n = 0; n < want_tiles + 40; ++n) {
                inside(a, t.seq, t.head, t.s, t.row0, t.n_rows, t.vis, "tiles");
                if (!moving && n < want_tiles && t.n_rows < 1) ++errors, std::printf("tiles: %ld items of %ld\n", n, want_tiles);
                if (!moving && n >= want_tiles && t.n_rows > 0) ++errors, std::printf("tiles: more than %ld\n", want_tiles);
                next_tile_item(a, 128, t);
            }
        }
    }
    return errors != 0;
}
"""


def read(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def block(text, start):
    """From `start` to the bracket that closes its first one."""
    at = text.index(start)
    i = text.index("{", at)
    depth = 0
    while True:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            return text[at:i] + (";" if start.startswith("struct") else "") + "\n"


def test_items_stay_inside_the_arrays(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    shared, rows, tiles = read("memq_attn.cuh"), read("memq_attn_paged.cu"), read("memq_attn_tiles.cuh")
    constants = "".join(re.findall(r"constexpr int (?:kRows|kKeys|kStart) = [^\n]*\n", rows)[:3])
    constants += "".join(re.findall(r"constexpr int (?:kTileKeys)[^\n]*\n|constexpr int kTileStart[^\n]*\n", tiles))
    source = constants + block(shared, "struct AttnSeq {") + block(shared, "__device__ __forceinline__ AttnSeq attn_seq(")
    source += block(rows, "__host__ __device__ constexpr int tiles_of" if "constexpr int tiles_of" in rows
                    else "__device__ __forceinline__ int tiles_of(") + block(rows, "struct RowItem {")
    source += block(tiles, "struct TileItem {") + block(tiles, "__device__ __forceinline__ void tile_sizes(")
    source += block(tiles, "__device__ __forceinline__ bool tile_served(")
    source += block(tiles, "__device__ __forceinline__ void next_tile_item(")
    src, exe = tmp_path / "items.cpp", tmp_path / "items"
    src.write_text(PROGRAM.replace("SOURCE", source))
    subprocess.check_call([cxx, "-O1", "-std=c++17", "-x", "c++", str(src), "-o", str(exe)])
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout[:2000]


def test_notes_and_first_items_of_lengths_that_change():
    """An item's note goes to one of the runs' places, and the tensor-core kernel's first item is none until a thread has
    found it."""
    rows = re.sub(r"//[^\n]*", "", read("memq_attn_paged.cu"))
    rows = rows[rows.index("attn_rows_kernel(const __grid_constant__"):rows.index("struct JoinPart")]
    notes = [m.start() for m in re.finditer(r"a\.owner\[(?!run\])", rows)]
    assert len(notes) == 2 and all("it.index < runs" in rows[at - 80:at] for at in notes)
    tiles = re.sub(r"//[^\n]*", "", read("memq_attn_tiles.cuh"))
    body = tiles[tiles.index("attn_tiles_kernel(const AttnArgs a)"):]
    assert body.index("ctl->first = TileItem{};") < body.index("__syncthreads") < body.index("ctl->first = it;")
    assert body.index("ctl->first_off = 0;") < body.index("__syncthreads")
    assert body.index("ctl->first_pos = 1ll << 62;") < body.index("__syncthreads")

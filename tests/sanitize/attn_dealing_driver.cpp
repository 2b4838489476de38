// Host-only driver for the attention's shapes and dealing, built with AddressSanitizer and
// UndefinedBehaviorSanitizer from the library's own sources: bpw_decode_host.cpp (the shape of a call)
// and bpw_decode.h (the dealing that the kernels compute from it). The launchers are stubs that
// abort if reached.
//
// Each argument is one call, "n_tokens,n_seqs,max_q,q_heads,kv_heads,head_dim,prefix_len,page_size,max_pages:len x tokens,..."
// with the sequences' lengths and query tokens ("122880x1,0x1"). Output, one line per argument:
//   "<status> <mp> <ms> <workgroups> <most parts of a query row> <most parts a row may have> <one launch>"
// after checking that every run is one wave's, that the runs hold all units, and that every (item, run) has a part of
// its own inside the workspace.
#include "../../bit_plane_weight_amd/csrc/bpw_decode_host.cpp"

#include <cstdlib>
#include <set>
#include <vector>

[[noreturn]] static void unreachable(const char *what) {
    std::fprintf(stderr, "dealing driver: %s reached\n", what);
    std::abort();
}
extern "C" const char *hipGetErrorString(hipError_t) { unreachable("hipGetErrorString"); }
namespace bpw {
void record_error(const char *) {}
int host_check_device() { unreachable("host_check_device"); }
int launch_heads(const HeadsArgs &, int32_t, int32_t, int32_t, void *) { unreachable("a launcher"); }
int launch_attn_d64(const AttnArgs &, int32_t, int32_t, int32_t, void *) { unreachable("a launcher"); }
int launch_attn_d128(const AttnArgs &, int32_t, int32_t, int32_t, void *) { unreachable("a launcher"); }
int launch_attn_d256(const AttnArgs &, int32_t, int32_t, int32_t, void *) { unreachable("a launcher"); }
int launch_verify(const VerifyArgs &, int32_t, void *) { unreachable("a launcher"); }
}  // namespace bpw

static void require(bool ok, const char *what) {
    if (ok) return;
    std::fprintf(stderr, "dealing driver: %s\n", what);
    std::exit(1);
}

int main(int argc, char **argv) {
    static uint16_t memory[8];
    for (int x = 1; x < argc; ++x) {
        int v[9], at = 0;
        const char *p = argv[x];
        for (int &y : v) {
            require(std::sscanf(p, "%d%n", &y, &at) == 1, "bad argument");
            p += at + 1;
        }
        std::vector<int> lens, toks;
        for (int l, t; std::sscanf(p, "%dx%d%n", &l, &t, &at) == 2;) {
            lens.push_back(l);
            toks.push_back(t);
            p += at;
            if (*p++ != ',') break;
        }
        bpw_attn_shared_prefix_args a{};
        a.n_tokens = v[0], a.n_seqs = v[1], a.max_q = v[2], a.q.heads = v[3], a.prefix_len = v[6], a.max_pages = v[8];
        a.kv.kv_heads = v[4], a.kv.head_dim = v[5], a.kv.page_size = v[7], a.kv.n_pages = 1;
        a.kv.dtype = BPW_BF16;
        a.kv.d_k = a.kv.d_v = memory;
        a.kv.k_row_stride = a.kv.v_row_stride = v[5];
        AttnShape s{};
        const bpw_status st = attn_shape(&a, &s);
        if (st) {
            std::printf("%d 0 0 0 0 %d 0\n", st, bpw::kAttnParts);
            continue;
        }
        require((int)lens.size() == v[1], "sequences");
        const int64_t unit = s.mp > 32 ? bpw::kWideTile : bpw::kAttnStep;
        const int up = (int)((a.prefix_len + unit - 1) / unit), total_p = a.kv.kv_heads * s.tiles_p * up;
        std::vector<int> units(1, 0), items(1, 0);
        for (int b = 0; b < v[1]; ++b) {
            const int64_t len = lens[b] < s.cap ? lens[b] : s.cap;
            const int u = (int)((len + bpw::kAttnStep - 1) / bpw::kAttnStep);
            const int it = u > 0 ? a.kv.kv_heads * ((toks[b] * s.group + s.ms - 1) / s.ms) : 0;
            units.push_back(units.back() + it * u);
            items.push_back(items.back() + it);
        }
        const int total_s = units.back(), waves = bpw::kAttnWaves * s.n_wgs;
        bpw::AttnDeal d;
        int runs = waves;  // of the suffixes
        int most_p = 0, most_s = 0;
        if (s.mp > 32) {
            const int pieces = a.kv.kv_heads * s.tiles_p * s.splits, per = (pieces + 7) / 8, wgs = s.n_wgs / 8;
            const int turns = (per + wgs - 1) / wgs, busy = per - (turns - 1) * wgs, idle = 8 * (wgs - busy);
            d = bpw::deal_wide(total_s, items.back(), idle, s.split_units, s.mp == 64, s.n_wgs);
            most_p = s.splits;
            require(pieces <= s.pieces_p && (int64_t)s.splits * s.split_units >= up, "pieces");
            std::set<int> seen;  // the run of each wave
            for (int block = 0; block < s.n_wgs; ++block)
                for (int wave = 0; wave < bpw::kAttnWaves; ++wave)
                    seen.insert(bpw::wide_run(block, wave, busy, idle));
            require((int)seen.size() == waves && *seen.begin() == 0 && *seen.rbegin() == waves - 1, "a wave to each run");
        } else {
            d = bpw::deal_narrow(total_p, total_s, s.n_wgs);
            runs = waves - d.wp;
            for (int item = 0; up > 0 && item < a.kv.kv_heads * s.tiles_p; ++item) {
                const int w0 = item * up / d.qb, n = (item * up + up - 1) / d.qb - w0 + 1;
                most_p = n > most_p ? n : most_p;
                require(item + w0 + n <= s.pieces_p && w0 + n <= d.wp, "a part inside the workspace (prefix)");
            }
        }
        require(total_s == 0 || d.run_of(total_s - 1) < runs, "all units dealt");
        int64_t last = -1;
        for (int b = 0; b < v[1]; ++b) {
            const int n = items[b + 1] - items[b], ub = n ? (units[b + 1] - units[b]) / n : 0;
            for (int i = 0; i < n; ++i) {
                const int w0 = d.run_of(units[b] + i * ub), w1 = d.run_of(units[b] + i * ub + ub - 1);
                const int64_t first = (int64_t)items[b] + i + w0;
                require(first > last && first - w0 + w1 < s.pieces_s, "a part inside the workspace, and its own");
                last = first - w0 + w1;
                most_s = w1 - w0 + 1 > most_s ? w1 - w0 + 1 : most_s;
            }
        }
        std::printf("%d %d %d %d %d %d %d\n", st, s.mp, s.ms, s.n_wgs, most_p + most_s, bpw::kAttnParts, s.one_launch);
    }
    return 0;
}

// The gradients beside a microscaled matrix: dY's planes, tile choice, tensor
// maps.
#include "mx_grad.cuh"
#include "mx_units.h"

namespace sgemm_gb300 {
namespace units {

// The tile of rows p and the split of the contraction that an estimate of the
// time prefers: per stage the largest of the MMA's cycles (2 BN a plane), the
// traffic of its CTA's shared memory at 128 bytes a cycle (dY's rows and the codes,
// written and read), the loads at ~52 bytes a cycle and the decoding (550); per
// tile a start and a drain, which a single accumulator (256 rows) does not hide,
// per cluster its exchange.  Of 66 sizes with all choices timed (16 to 8192 rows,
// FP32 and bfloat16, 4 and 8 bits) the one taken was within 3 % of the best.
MxPlan mx_grad_plan(int p, int c, long long stages, int bits, bool transposed, bool f32, const MxDevice &d) {
    const long long tiles_c = ((long long)c + mx::TC_M - 1) / mx::TC_M;
    const int planes = f32 ? 3 : 1;
    MxPlan best = {16, 1, false};
    double best_cost = 1e300;
    for (int bn : {16, 64, 128, 256}) {
        if ((transposed && bn < 64) || (f32 && bn > 128)) continue;
        const long long tiles_p = ((long long)p + bn - 1) / bn;
        for (bool pair : {false, true}) {
            // 256 rows, and 128 of FP32, come as pairs' tiles alone, 64 of FP32 both ways; 64
            // transposed rows are a box of dY, which a pair cannot halve
            if (pair ? bn < (f32 && !transposed ? 64 : f32 ? 128 : 256) : bn == 256 || (f32 && bn == 128)) continue;
            const long long tiles = pair ? (tiles_c + 1) / 2 * tiles_p : tiles_c * tiles_p;
            const double rows = mx::g_x_bytes(pair ? bn / 2 : bn), raw = mx::g_raw_bytes(bits);
            const double traffic = (2 * planes * rows + 2 * raw) / 128.0, bytes = (planes * rows + raw) / 52.0;
            double stage = 2.0 * bn * planes;
            for (double other : {traffic, bytes, 550.0})
                if (stage < other) stage = other;
            for (int s = 1; s <= (pair ? 1 : 8); ++s) {
                if (s > 1 && (tiles > d.clusters[s] || stages < 2 * s)) continue;
                const long long fit = pair ? d.sms / 2 : d.sms, waves = s > 1 ? 1 : (tiles + fit - 1) / fit;
                const double cost = (double)waves * ((double)((stages + s - 1) / s) * stage + (bn == 256 ? 1500.0 : 300.0)) + 1700.0 + 4.0 * bn + (s > 1 ? 500.0 + 32.0 * bn : 0.0);
                if (cost < best_cost) {
                    best_cost = cost;
                    best = {bn, s, pair};
                }
            }
        }
        if (bn >= p) break;
    }
    return best;
}

cudaError_t mx_grad_setup() {
    cudaError_t e = mx_grad4_setup();
    return e != cudaSuccess ? e : mx_grad8_setup();
}

cudaError_t mx_planes(const mx::PlaneArgs &a, bool f32, int sms, cudaStream_t s) {
    const long long warps = (long long)a.rows * (a.cols / 256 + (a.cols % 256 != 0)), ctas = (warps + mx::PLANE_THREADS / 32 - 1) / (mx::PLANE_THREADS / 32),
                    most = (long long)sms * 8;
    return launch_early(f32 ? mx::planes_kernel<float> : mx::planes_kernel<__nv_bfloat16>, dim3((unsigned)(ctas < most ? ctas : most)), mx::PLANE_THREADS, 0, a, s);
}

size_t mx_grad_sums_bytes(const GradCall &g, bool f32, const MxDevice &d) {
    const long long stages = ((long long)g.depth + mx::G_K - 1) / mx::G_K;
    if (f32 || stages <= mx::G_DEEP) return 0;
    const MxPlan p = mx_grad_plan(g.out.rows, g.out.cols, stages, g.bits, g.transposed, f32, d);
    return mx_sums_bytes(p, g.out.rows, g.out.cols, (stages + p.split - 1) / p.split, mx::G_DEEP, d);
}

cudaError_t mx_grad(const GradCall &g, const MxDevice &d, cudaStream_t s) {
    mx::GradArgs a = {g.out, g.depth, 0, 0, 0, g.sums};
    const int p_rows = g.out.rows, cols = g.out.cols;
    const bool f32 = g.planes == 3;
    const long long stages = ((long long)g.depth + mx::G_K - 1) / mx::G_K;
    const MxPlan p = mx_grad_plan(p_rows, cols, stages, g.bits, g.transposed, f32, d);
    const MxGrid grid = mx_grid(p, p_rows, cols, d);
    const int ctas = p.pair ? 2 : p.split, rows = p.pair ? p.bn / 2 : p.bn;
    a.tiles_c = grid.tiles_f;
    a.tiles_p = grid.tiles_r;
    a.group = p.pair ? 8 : 16;
    CUtensorMap m[3];
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int nb = mx::blocks(cols);
    cudaError_t e = mx_map(&m[0], u8, 1, g.codes, (long long)nb * mx::block_bytes(g.bits), g.depth, g.ldc, mx::TC_M * g.bits / 8, mx::G_K, true);
    if (e == cudaSuccess) e = mx_map(&m[1], u8, 1, g.scales, nb, g.depth, g.lds, 16, mx::G_K, false);
    const int inner = g.transposed ? p_rows : g.depth, outer = g.transposed ? g.depth : p_rows;
    if (e == cudaSuccess) e = mx_map3(&m[2], g.dy, inner, outer, g.planes, g.lddy, g.plane, 64, g.transposed ? mx::G_K : rows);
    if (e != cudaSuccess) return e;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid.clusters * ctas), 1, 1);
    cfg.blockDim = dim3((unsigned)mx::G_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)mx::g_smem_bytes(p.bn, p.pair, g.bits, f32);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    unsigned na = 0;
    if (ctas > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = (unsigned)ctas;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    cfg.attrs = attr;
    cfg.numAttrs = na;
    return g.bits == 4 ? mx_grad4_launch(cfg, p, g.transposed, f32, m, a) : mx_grad8_launch(cfg, p, g.transposed, f32, m, a);
}

cudaError_t mx_grad_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300

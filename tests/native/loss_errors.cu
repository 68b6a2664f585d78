// Test program (not part of the library): what the loss' calls leave behind when a kernel of theirs has reported an error.
// No wait is made to run out: the error word of the workspace is set between a call's kernels, which are launched here one by
// one from the library's source.
#include "zero_lm_loss.cu"

#include <cstdio>
#include <vector>

namespace {

bool is_nan(uint16_t bf16) { return (bf16 & 0x7F80) == 0x7F80 && (bf16 & 0x7F); }

int failures = 0;

void expect(bool ok, const char* what, int n, int d) {
    if (ok) return;
    ++failures;
    printf("n %d, d %d: %s\n", n, d, what);
}

template <class T>
T* upload(const std::vector<T>& v) {
    T* p = nullptr;
    if (cudaMalloc(&p, v.size() * sizeof(T)) != cudaSuccess) exit(2);
    cudaMemcpy(p, v.data(), v.size() * sizeof(T), cudaMemcpyHostToDevice);
    return p;
}

template <class T>
std::vector<T> download(const T* p, size_t n) {
    std::vector<T> v(n);
    if (cudaMemcpy(v.data(), p, n * sizeof(T), cudaMemcpyDeviceToHost) != cudaSuccess) exit(3);
    return v;
}

void run(int n, int d, int vocab, bool set_error) {
    std::vector<uint16_t> h(n * d), w(vocab * d);
    for (int i = 0; i < n * d; ++i) h[i] = (uint16_t)(0x3F00 + i * 37 % 64 + (i * 11 % 2 << 15));   // 0.5 .. 0.75 in bf16, both signs
    for (int i = 0; i < vocab * d; ++i) w[i] = (uint16_t)(0x3E00 + i * 53 % 64 + (i * 7 % 2 << 15));
    std::vector<int64_t> t(n);
    for (int i = 0; i < n; ++i) t[i] = i % 5 == 4 ? -1 : i * 3 % vocab;
    std::vector<uint16_t> zeros(std::max(n, vocab) * d, 0);
    zero_lm_loss_args a{};
    a.n = n, a.d = d, a.vocab = vocab, a.hidden_stride = d, a.dtype = ZERO_BF16, a.reduction = ZERO_LOSS_MEAN, a.scale = 1.0;
    uint16_t *gh = upload(zeros), *gw = upload(zeros);
    a.hidden = upload(h), a.weight = upload(w), a.targets = upload(t);
    a.losses = upload(std::vector<float>(n)), a.lse = upload(std::vector<float>(n)), a.stats = upload(std::vector<float>(2));
    int64_t fb = 0, bb = 0;
    if (zero_lm_loss_query(&a, &fb, &bb) != ZERO_OK) exit(4);
    a.workspace = upload(std::vector<uint8_t>(std::max(fb, bb)));
    if (zero_lm_loss_forward(&a, nullptr) != ZERO_OK || cudaDeviceSynchronize() != cudaSuccess) exit(5);
    const LossPlan p = make_plan(&a);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    zk::LossHead head = download(reinterpret_cast<zk::LossHead*>(ws), 1)[0];
    head.error = set_error ? zk::ZERO_DEVERR_WAIT_TIMEOUT : 0;
    head.ticket = 0;
    cudaMemcpy(ws, &head, sizeof head, cudaMemcpyHostToDevice);
    zk::LossArgs l{};   // as zero_lm_loss_forward fills it
    l.head = reinterpret_cast<zk::LossHead*>(ws);
    l.parts = reinterpret_cast<const float2*>(ws + p.parts);
    l.ld = p.part_ld;
    l.tiles = (int32_t)p.part_ld;
    l.blocks = (n + zk::kLossRows - 1) / zk::kLossRows;
    l.z_target = reinterpret_cast<const float*>(ws + p.z_target);
    l.token = reinterpret_cast<const int32_t*>(ws + p.token);
    l.losses = a.losses, l.lse = a.lse, l.stats = a.stats;
    l.block_sums = reinterpret_cast<double*>(ws + p.sums);
    zk::loss_kernel<<<l.blocks, zk::kThreads>>>(l);
    const std::vector<float> stats = download(a.stats, 2);
    expect(std::isnan(stats[0]) == set_error, "the loss", n, d);
    int32_t bits = -1;
    expect(zero_lm_loss_device_error(ws, &bits) == ZERO_OK && bits == head.error, "the workspace's report", n, d);
    // the backward call, whose own kernels report nothing
    a.grad_hidden = gh, a.grad_weight = gw;
    if (zero_lm_loss_backward(&a, nullptr) != ZERO_OK || cudaDeviceSynchronize() != cudaSuccess) exit(6);
    expect(zero_lm_loss_device_error(ws, &bits) == ZERO_OK && bits == 0, "the backward call's report", n, d);
    std::vector<uint16_t> x = download(gh, n * d), y = download(gw, vocab * d);
    bool hidden = true, weight = true;
    for (int i = 0; i < n * d; ++i) hidden = hidden && is_nan(x[i]) == (set_error && t[i / d] >= 0);
    for (uint16_t e : y) weight = weight && is_nan(e) == set_error;
    expect(hidden, "grad_hidden after the forward call's error", n, d);
    expect(weight, "grad_weight after the forward call's error", n, d);
    // an error of the backward call's own kernels: its last one marks the first rows of whichever gradients there are
    const uint16_t nan = 0x7FC0;
    for (int which = 0; which < 4; ++which) {
        cudaMemset(gh, 0, n * d * 2);
        cudaMemset(gw, 0, vocab * d * 2);
        head.error = set_error ? zk::ZERO_DEVERR_WAIT_TIMEOUT : 0;
        cudaMemcpy(ws, &head, sizeof head, cudaMemcpyHostToDevice);
        const zk::VerdictArgs v{reinterpret_cast<zk::LossHead*>(ws), which & 1 ? gh : nullptr, which & 2 ? gw : nullptr, (uint32_t)d, nan};
        zk::verdict_kernel<<<1, 32>>>(v);
        x = download(gh, n * d), y = download(gw, vocab * d);
        bool marked = true;
        for (int i = 0; i < n * d; ++i) marked = marked && x[i] == (set_error && (which & 1) && i < d ? nan : 0);
        for (int i = 0; i < vocab * d; ++i) marked = marked && y[i] == (set_error && (which & 2) && i < d ? nan : 0);
        expect(marked, "the rows that the last kernel marks", n, d);
    }
    const void* all[] = {gh, gw, a.hidden, a.weight, a.targets, a.losses, a.lse, a.stats, a.workspace};
    for (const void* q : all) cudaFree(const_cast<void*>(q));
}

}  // namespace

int main() {
    // one CTA's tiles and pairs', rows that the products write themselves and such that finish_kernel writes
    const int shapes[][3] = {{5, 16, 40}, {5, 24, 40}, {1, 8, 3}, {300, 32, 500}, {300, 24, 77}, {4000, 256, 600}};
    for (const auto& s : shapes)
        for (bool set_error : {false, true}) run(s[0], s[1], s[2], set_error);
    printf("failures=%d cuda=%d\n", failures, (int)cudaDeviceSynchronize());
    return failures;
}
